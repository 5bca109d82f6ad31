"""Launch limits and workspaces of the layer calls at their borders: refused with a reason before a device is looked for."""
import ctypes

import pytest

from test_layer_errors import INVALID, MANY, L, norm_desc, refused  # noqa: F401

ROWS = [(8, 2 ** 29 - 32), (64, 2 ** 29 - 32), (72, 2 ** 28 - 16), (128, 2 ** 28 - 16), (136, 2 ** 27 - 8), (256, 2 ** 27 - 8),
        (264, 2 ** 26 - 4), (512, 2 ** 26 - 4), (520, 2 ** 24 - 1), (8192, 2 ** 24 - 1), (8200, 2 ** 22 - 1), (32768, 2 ** 22 - 1)]


def good(L, rc):  # noqa: F811
    """Accepted: without a GPU such a call gets as far as looking for one, and with one this is not asked."""
    refused(L, rc, INVALID, "device 0 not available")


@pytest.mark.parametrize("d,most", ROWS)
def test_rows_of_the_norm(L, d, most):  # noqa: F811
    torch = pytest.importorskip("torch")
    n = ctypes.c_size_t()
    for heads in (1, 4):
        for out in (1, 3):
            over = ctypes.byref(norm_desc(n_rows=most // heads + 1, n_heads=heads, d=d, out_dtype=out))
            refused(L, L.stepq_norm_forward(over, *MANY[:7], None), INVALID, "launch grid")
            if not torch.cuda.is_available():
                fits = ctypes.byref(norm_desc(n_rows=most // heads, n_heads=heads, d=d, out_dtype=out))
                good(L, L.stepq_norm_forward(fits, *MANY[:7], None))
        over = ctypes.byref(norm_desc(n_rows=most // heads + 1, n_heads=heads, d=d))
        rc = L.stepq_norm_backward_workspace(over, ctypes.byref(n))
        if d > 512:
            refused(L, rc, INVALID, "launch grid")
        else:
            assert rc == 0


@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_columns_of_the_scans_last_sums(L, n):  # noqa: F811
    from test_layer_errors import scan_desc
    size = ctypes.c_size_t()
    most = (2 ** 28 - 64) // (n + 2) // 8 * 8
    if most + 8 >= 2 ** 24:
        most = 2 ** 24 - 16  # other limits come first: every number of channels has its gradient
    for ch in (most, most + 8):
        d = ctypes.byref(scan_desc(channels=ch, n_groups=1, d_state=n, n_seqs=1, n_tokens=1))
        assert L.stepq_scan_forward_workspace(d, ctypes.byref(size)) == 0
        rc = L.stepq_scan_backward_workspace(d, ctypes.byref(size))
        if ch > most and most < 2 ** 24 - 16:
            refused(L, rc, INVALID, "gradient's launch grid")
            refused(L, L.stepq_scan_backward(d, *MANY[:21], 1 << 50, None), INVALID, "gradient's launch grid")
        else:
            assert rc == 0


def test_workspace_of_the_norms_gradient(L):  # noqa: F811
    """A row of partial sums for each workgroup that writes one, no more; none where dweight is not wanted."""
    torch = pytest.importorskip("torch")
    n = ctypes.c_size_t()
    for rows, d, groups in ((0, 64, 0), (1, 64, 1), (32, 64, 1), (33, 64, 2), (8192, 128, 512), (100000, 128, 1024), (5, 512, 2),
                            (7, 1024, 7), (2000, 2048, 1024), (2000, 2056, 512), (8192, 4096, 512), (600, 32768, 512), (9, 32768, 9)):
        desc = ctypes.byref(norm_desc(n_rows=rows, n_heads=1, d=d))
        assert L.stepq_norm_backward_workspace(desc, ctypes.byref(n)) == 0 and n.value == groups * d * 4, (rows, d)
        if rows:
            p = list(MANY[:8])
            refused(L, L.stepq_norm_backward(desc, *p, MANY[9], n.value - 1, None), INVALID, "workspace")
            p[6] = None
            if not torch.cuda.is_available():
                good(L, L.stepq_norm_backward(desc, *p, None, 0, None))


def test_workspaces_of_the_scan(L):  # noqa: F811
    """No more than the interface tells, for many short sequences, narrow groups and long sequences alike."""
    import random
    from test_layer_errors import scan_desc
    rng, size = random.Random(5), ctypes.c_size_t()
    calls = [(8192, 8192, 4096, 1, 16), (16384, 512, 4096, 512, 16), (16384, 1, 4096, 1, 16), (270000, 2, 8192, 1, 16), (0, 3, 64, 1, 8),
             (1, 1, 8, 1, 64), (4000, 200, 8, 1, 64)]
    for _ in range(400):
        G, N = rng.choice([1, 1, 2, 16, 64]), int(10 ** rng.uniform(0, 3.6))
        calls.append((int(10 ** rng.uniform(0, 5)), N, 8 * G * rng.randint(1, 40), G, rng.choice([8, 16, 32, 64])))
    for T, N, ch, G, n in calls:
        d = ctypes.byref(scan_desc(channels=ch, n_groups=G, d_state=n, n_seqs=N, n_tokens=T, cu_seqlens=4096))
        wide = G * ((ch // G + 31) // 32 * 32)
        cut = 13 * wide * n * N + max(14 * wide * n * N, 1.2e6 * n)
        assert L.stepq_scan_forward_workspace(d, ctypes.byref(size)) == 0 and size.value <= cut, (T, N, ch, G, n)
        assert L.stepq_scan_backward_workspace(d, ctypes.byref(size)) == 0
        assert size.value <= wide * n * (T / 2 + 9 * N) + cut + 4096, (T, N, ch, G, n)
