"""Host-side refusals of the dense operators (no GPU needed)."""
import ctypes

import pytest

import quantised_expert_decode_b200 as q
from quantised_expert_decode_b200 import _lib as L

FAKE = 1 << 20   # aligned non-null address; never dereferenced by the host checks below


def test_norm_argument_checks():
    lib = q.lib()

    def call(x=FAKE, y=FAKE, dt=q.F32, gain=FAKE, eps=1e-6, T=1, H=2048, group=0, z=FAKE, norm=None, codes=FAKE, scales=FAKE):
        return lib.qmoe_rmsnorm_residual_q8(x, y, dt, gain, ctypes.c_float(eps), T, H, group, z, norm, codes, scales, None)

    assert call(x=None) == 1 and call(T=0) == 1 and call(H=0) == 1 and call(dt=q.I8) == 1
    assert call(codes=None) == 1 and call(scales=None) == 1                     # codes and scales go together
    assert call(codes=None, scales=None) == 1                                   # nothing to write
    for name in ("x", "y", "gain", "z", "norm", "codes"):
        assert call(**{name: FAKE + 8}) == 1, name
    assert call(scales=FAKE + 2) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(H=2040) == 3 and call(H=16400) == 3
    assert call(group=16) == 3 and call(group=-32) == 3 and call(group=256) == 3 and call(group=128, H=2048 + 64) == 3


def test_quantise_argument_checks():
    lib = q.lib()

    def call(x=FAKE, dt=q.BF16, T=1, H=64, group=0, codes=FAKE, scales=FAKE):
        return lib.qmoe_quantise_rows(x, dt, T, H, group, codes, scales, None)

    assert call(x=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1 and call(T=0) == 1 and call(dt=5) == 1
    assert call(x=FAKE + 4) == 1 and call(codes=FAKE + 4) == 1 and call(scales=FAKE + 1) == 1
    assert call(H=24) == 3 and call(group=96) == 3 and call(H=32768) == 3


def test_linear_argument_checks():
    lib = q.lib()

    def call(a=FAKE, dt=q.BF16, w=FAKE, M=4, N=64, K=64, sa=None, sw=None, bias=None, act=0, res=None, out=FAKE,
             odt=q.F32, lda=0, ldw=0, ldr=0, ldo=0, st=FAKE):
        return lib.qmoe_linear(a, dt, w, M, N, K, sa, sw, bias, act, res, out, odt, lda, ldw, ldr, ldo, st, None)

    assert call(a=None) == 1 and call(w=None) == 1 and call(out=None) == 1 and call(st=None) == 1
    assert call(M=0) == 1 and call(N=0) == 1 and call(K=0) == 1 and call(M=-3) == 1
    assert call(dt=q.F32) == 1 and call(odt=q.I8) == 1 and call(act=4) == 1 and call(act=-1) == 1
    assert call(sa=FAKE) == 1 and call(dt=q.I8) == 1 and call(dt=q.I8, sa=FAKE) == 1       # scales: 8-bit only, both
    assert call(lda=63) == 1 and call(ldw=8) == 1 and call(ldo=63) == 1 and call(res=FAKE, ldr=60) == 1
    assert call(lda=-64) == 1
    for name in ("a", "w", "out", "bias", "res"):
        assert call(**{name: FAKE + 4}) == 1, name
    assert call(st=FAKE + 2) == 1
    assert call(K=60) == 3 and call(K=60, lda=64) == 3 and call(K=60, lda=64, ldw=61) == 3   # rows off 16 bytes
    assert call(K=72, dt=q.I8, sa=FAKE, sw=FAKE) == 3
    assert call(K=65536 + 64) == 3 and call(lda=1 << 40) == 3


def test_sample_argument_checks():
    lib = q.lib()

    def call(l=FAKE, dt=q.F32, T=2, V=100, ld=0, temp=None, k=None, p=None, mp=None, u=FAKE, tok=FAKE, prob=None, st=FAKE):
        return lib.qmoe_sample(l, dt, T, V, ld, temp, k, p, mp, u, tok, prob, st, None)

    assert call(l=None) == 1 and call(u=None) == 1 and call(tok=None) == 1 and call(st=None) == 1
    assert call(T=0) == 1 and call(V=0) == 1 and call(ld=99) == 1 and call(ld=-1) == 1 and call(dt=q.I8) == 1
    assert call(l=FAKE + 8) == 1
    for name in ("temp", "k", "p", "mp", "u", "tok", "prob", "st"):
        assert call(**{name: FAKE + 2}) == 1, name
    assert call(V=393217) == 3


def test_sizes_past_the_limits_are_refused():
    lib, F = q.lib(), FAKE
    assert lib.qmoe_rmsnorm_residual_q8(F, None, q.F32, None, ctypes.c_float(0), (1 << 30) + 1, 16, 0, None, None, F, F, None) == 3
    assert lib.qmoe_quantise_rows(F, q.F32, (1 << 30) + 1, 16, 0, F, F, None) == 3
    for M, N in (((1 << 30) + 1, 1), (1, (1 << 30) + 1)):
        assert lib.qmoe_linear(F, q.BF16, F, M, N, 8, None, None, None, 0, None, F, q.F32, 0, 0, 0, 0, F, None) == 3
    assert lib.qmoe_sample(F, q.F32, (1 << 27) + 1, 1, 0, None, None, None, None, F, F, None, F, None) == 3


def test_linear_strides_past_the_limit_are_refused():
    lib, F, big = q.lib(), FAKE, 1 << 62

    def call(lda=0, ldw=0, ldr=0, ldo=0):
        return lib.qmoe_linear(F, q.BF16, F, 2, 8, 8, None, None, None, 0, F, F, q.F32, lda, ldw, ldr, ldo, F, None)

    for name in ("lda", "ldw", "ldr", "ldo"):
        assert call(**{name: big}) == 3 and call(**{name: (1 << 37) + 8}) == 3, name


def test_linear_in_place_at_another_stride_is_refused():
    lib, F = q.lib(), FAKE

    def call(M, ldr, ldo, out):
        return lib.qmoe_linear(F, q.BF16, F, M, 8, 8, None, None, None, 0, F, out, q.F32, 0, 0, ldr, ldo, F, None)

    for ldr, ldo in ((16, 8), (0, 12), (8, 16)):
        assert call(2, ldr, ldo, F) == 1


@pytest.mark.gpu
def test_binding_refuses_a_status_word_off_the_device():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a device to be off of")
    st = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 64), device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(q.QmoeError):
        q.qmoe_sample(x, q.F32, 1, 64, None, None, None, None, x[0, :1], i, None, st)
    b = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(q.QmoeError):
        q.qmoe_linear(b, q.BF16, b, 1, 1, 64, None, None, None, 0, None, x, q.F32, st)


class _OnAnotherDevice:
    """Just enough of a tensor to be looked at."""

    import torch
    dtype = torch.float32

    def get_device(self):
        return 1


def test_binding_refuses_tensors_that_do_not_fit(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # CPU tensors report device -1
    x = torch.zeros(4, 64)
    f = "float32"
    L._fits("f", (x, f, 4, 64, 64), (x, f, 2, 64, 64), (None, f, 9, 9, 9), (123, f, 9, 9, 9))
    L._fits("f", (x[:, :50], f, 4, 50, 64), (x[1:], f, 3, 64, 64))
    for bad in ((x, f, 5, 64, 64), (x[1:], f, 4, 64, 64), (x.t(), f, 4, 64, 64), (x[:, :50], f, 4, 50, 50),
                (x, "bfloat16", 4, 64, 64), (x.double(), f, 4, 64, 64), (_OnAnotherDevice(), f, 1, 1, 0)):
        with pytest.raises(q.QmoeError):
            L._fits("f", bad)


def _fits_on_cpu(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # CPU tensors report device -1
    return torch, "float32"


def test_binding_refuses_rows_that_are_not_at_one_stride(monkeypatch):
    """Views whose rows do not follow one another at the stride that the call reads with."""
    torch, f = _fits_on_cpu(monkeypatch)
    h = torch.zeros(4, 8, 64)
    bad = {"last position of each sequence": (h[:, -1:, :], f, 4, 64, 64),
           "the same, squeezed": (h[:, -1], f, 4, 64, 64),
           "two positions of each sequence": (h[:, :2], f, 8, 64, 64),
           "heads apart": (torch.zeros(4, 2, 96)[:, :, :64], f, 8, 64, 64),
           "transposed heads": (torch.zeros(2, 4, 64).transpose(0, 1), f, 8, 64, 64),
           "broadcast rows": (torch.zeros(1, 64).expand(4, 64), f, 4, 64, 64),
           "narrower rows than the call's": (torch.zeros(4, 32), f, 2, 64, 64),
           "a column of rows": (torch.zeros(6, 4)[:, :1], f, 1, 6, 0),
           "a column": (torch.zeros(6, 4)[:, 1], f, 1, 6, 0),
           "packed scales in wider rows": (torch.zeros(6, 10)[:, :4], f, 1, 24, 0),
           "one value broadcast": (torch.zeros(1).expand(6), f, 1, 6, 0)}
    for name, want in bad.items():
        with pytest.raises(q.QmoeError):
            L._fits("f", want)
            pytest.fail(name)
    for good in ((h, f, 32, 64, 64), (h[1], f, 8, 64, 64), (h[1:3], f, 16, 64, 64), (h[:1, -1:, :], f, 1, 64, 64),
                 (h[:, -1], f, 4, 64, 512), (h[:, -1:, :], f, 4, 64, 512), (h.view(-1), f, 32, 64, 64),
                 (h.view(-1), f, 4, 64, 500), (h.view(32, 64)[:, :50], f, 32, 50, 64), (h.view(32, 64), f, 32, 50, 64),
                 (torch.zeros(6, 1), f, 1, 6, 0), (torch.zeros(1, 6, 1), f, 1, 6, 0), (torch.zeros(6, 4), f, 1, 24, 0),
                 (torch.zeros(8, 1)[2:], f, 1, 6, 0), (torch.zeros(3, 1, 5)[1], f, 1, 5, 0),
                 (torch.zeros(6, 4)[2, :1], f, 1, 1, 0), (torch.nn.Parameter(torch.zeros(4, 64)), f, 4, 64, 64)):
        assert L._fits("f", good) == [good[0].data_ptr()]


def test_binding_refuses_views_shorter_than_the_call(monkeypatch):
    """What lies behind a view in its storage belongs to someone else."""
    torch, f = _fits_on_cpu(monkeypatch)
    x, u = torch.zeros(16, 64), torch.zeros(12)
    for bad in ((x[:2], f, 4, 64, 64), (x[:2, :50], f, 4, 50, 64), (x[:4, :40], f, 4, 50, 64), (u[:2], f, 1, 6, 0),
                (u[:0], f, 1, 1, 0), (x.view(-1)[:200], f, 4, 64, 64), (x[:4, :50], f, 5, 50, 64), (u[:0], f, 1, 6, 0)):
        with pytest.raises(q.QmoeError):
            L._fits("f", bad)
    L._fits("f", (x[:4], f, 4, 64, 64), (u[:6], f, 1, 6, 0), (x[:4, :50], f, 4, 50, 64), (x.view(-1)[:192 + 50], f, 4, 50, 64))


def test_token_head_refuses_hidden_states_of_scattered_rows(monkeypatch):
    torch, f = _fits_on_cpu(monkeypatch)
    from quantised_expert_decode_b200.model import TokenHead
    head = TokenHead.__new__(TokenHead)
    head.T, head.H, head.gain, head.eps, head.bits, head.norm = 4, 64, None, 1e-6, 8, None
    head.codes, head.scale = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    h = torch.zeros(4, 8, 64)
    for x in (h[:, -1:, :], h[:, -1], h[:, ::8]):
        with pytest.raises(q.QmoeError, match="row"):
            head.step(x, torch.zeros(4))
