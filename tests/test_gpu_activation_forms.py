"""Activation operators: forms that the sizes of the other tests do not reach."""
import numpy as np
import pytest
import torch

from oracle import activation as A
from tests.test_gpu_activation import DEV, DT, U, _params, draw, f64, strided
from tests.test_gpu_activation_large import _wgrad64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


@pytest.mark.parametrize("T,d", [(40, 264), (1500, 264), (40, 2056)])
def test_norm_rows_side_by_side(fw, T, d):
    """Inputs and outputs as column ranges of one buffer share no element: the
    same bits as from buffers of their own."""
    x, dy = draw(T, d, torch.bfloat16, 1), draw(T, d, torch.bfloat16, 2)
    w, b = _params(d, "bf16", "layer", "same", 3)
    y, mean, rstd = fw.norm_forward(x, w, b)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w)
    buf = torch.zeros(T, 4 * d + 8, dtype=torch.bfloat16, device=DEV)
    vx, vdy, vy, vdx = (buf[:, i * d:(i + 1) * d] for i in range(4))
    vx.copy_(x)
    vdy.copy_(dy)
    y2, mean2, rstd2 = fw.norm_forward(vx, w, b, out=vy)
    dx2, dw2, db2 = fw.norm_backward(vdy, vx, mean2, rstd2, w, dx=vdx)
    assert torch.equal(y2, y) and torch.equal(dx2, dx) and torch.equal(rstd2, rstd)
    # (rows that meet in memory take the columns in a launch of their own: the same sums)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)
    assert torch.equal(vx, x) and torch.equal(vdy, dy) and (buf[:, 4 * d:] == 0).all()
    with pytest.raises(fw.GiftError):
        fw.norm_forward(vx, w, b, out=buf[:, 8:8 + d])


# -- weight gradients of 256 x 256 tiles whose tokens are split over workgroups ----
# Pieces of 128 x 128 tiles need less than 64 MiB whatever the sizes (at most
# 1020 of them, 64 KiB each), so a larger workspace says which form runs.

def _large_split(fw, T, m, d, dtype):
    need = fw._lib.gift_weight_grad_workspace_bytes(T, m, d, fw.DTYPES[DT[dtype]])
    assert need > 64 << 20, "this size is to be computed in pieces of 256 x 256 tiles: take another"


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,m,d,ld,off", [(8192, 1024, 4096, None, 0), (8201, 1021, 4090, 1023, 1),
                                          (1000, 1533, 6130, 1535, 1)])     # (bf16: whole tiles, cut at both edges)
def test_weight_grad_large_tiles(fw, T, m, d, ld, off, dtype, fmt):
    """Against 64 bits; fp32 chains of at most T / 4 + 64 additions."""
    print(f"[wgrad T {T} {m}x{d} ld {ld} off {off} {dtype} {fmt}]", flush=True)
    if T > 8000:
        _large_split(fw, T, m, d, dtype)
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV).save(draw(T, d, torch.bfloat16, T + d))
    if T % 8:
        ck.bscales[-1, :, T % 8:] = 255
    delta = draw(T, m, DT[dtype], T + m, 0.01, ld, off)
    W = strided(m, d, torch.float32, d + 5, 3)
    fw.weight_grad(delta, ck, alpha=1.0 / T, out=W)
    ref, mag = _wgrad64(delta, ck, 1.0)
    alpha = float(np.float32(1.0 / T))
    assert ((W.double() - alpha * ref).abs() <= (T / 4 + 64) * U * alpha * mag + 1e-37).all()
    mask = torch.ones_like(W._base, dtype=torch.bool)
    torch.as_strided(mask, W.shape, W.stride(), W.storage_offset()).fill_(False)
    assert (W._base[mask] == 777.0).all()
    old = W.double()
    fw.weight_grad(delta, ck, alpha=0.25, out=W, accumulate=True)
    assert ((W.double() - 0.25 * ref - old).abs() <= (T / 4 + 64) * U * (0.25 * mag + old.abs()) + 1e-37).all()
    assert (W._base[mask] == 777.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_weight_grad_nonfinite_in_large_split_tiles(fw, dtype, fmt):
    T, m, d = 8192, 1024, 4096
    _large_split(fw, T, m, d, dtype)
    x = draw(T, d, torch.float32, 3)
    x[8190, 3000] = float("nan")
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV).save(x)
    delta = draw(T, m, DT[dtype], 4)
    delta[3, 700], delta[8191, 1000] = -float("inf"), float("nan")
    W = fw.weight_grad(delta, ck)
    bad = torch.zeros(m, d, dtype=torch.bool, device=DEV)
    bad[:, 3000 // 32 * 32:3000 // 32 * 32 + 32] = True
    bad[700] = bad[1000] = True
    assert torch.equal(~torch.isfinite(W), bad)
    # an infinity times a finite value keeps its sign
    a = ck.restore(torch.float32)[3]
    ok = torch.isfinite(a) & (a != 0) & ~bad[0]
    assert ok.sum() > d - 40 - (a == 0).sum() and (W[700][ok] == -torch.sign(a[ok]) * float("inf")).all()


def _one_token_a_column(fw, T, m, d, dtype, fmt, scale, seed):
    """delta and checkpoint for which each output is one product: column j of
    the activation is not zero at one token alone, where it is a power of two,
    and delta has all the bits its type holds (odd integers times scale)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    bits = {"bf16": 8, "fp16": 11, "fp32": 24}[dtype]
    toks = torch.randperm(T, generator=g, device=DEV)[:59]
    toks[0], toks[1] = 0, T - 1
    tok = toks[torch.arange(d, device=DEV) % toks.numel()]
    x = torch.zeros(T, d, device=DEV)
    pw = torch.randint(-3, 4, (d,), generator=g, device=DEV)
    x[tok, torch.arange(d, device=DEV)] = torch.exp2(pw.double()).float()
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV).save(x)
    assert torch.equal(ck.restore(torch.float32), x)
    n = torch.randint(1 << (bits - 2), 1 << (bits - 1), (T, m), generator=g, device=DEV) * 2 + 1
    n = torch.where(torch.rand(T, m, generator=g, device=DEV) < 0.5, -n, n)
    delta = (n.double() * scale).to(DT[dtype])
    assert torch.equal(delta.double(), n.double() * scale)
    return delta, ck, delta.double()[tok].t() * x.double()[tok, torch.arange(d, device=DEV)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,m,d", [(8201, 1021, 4090), (2048, 512, 2048), (700, 1530, 2100)])
def test_weight_grad_keeps_all_bits_in_every_form(fw, T, m, d, dtype, fmt):
    """Every sum is exact whatever the order, so W is, to the last of delta's bits."""
    if T > 8000:
        _large_split(fw, T, m, d, dtype)
    delta, ck, want = _one_token_a_column(fw, T, m, d, dtype, fmt, 1.0, T + m)
    W = fw.weight_grad(delta, ck)
    assert torch.equal(W.double(), want)
    fw.weight_grad(delta, ck, out=W, accumulate=True, alpha=-1.0)
    assert (W == 0).all()


@pytest.mark.parametrize("T,m,d", [(8201, 1021, 4090), (2048, 512, 2048), (64, 4, 64)])
def test_weight_grad_of_tiny_gradients(fw, T, m, d):
    """fp32 gradients whose last bit is 2^-133, the smallest bf16 number, lose
    nothing.  Of smaller ones the matrix-core form (m >= 8) drops what lies
    below that bit: less than 2^-133 for each, times the activation."""
    delta, ck, want = _one_token_a_column(fw, T, m, d, "fp32", "e4m3", 2.0 ** -133, 5)
    assert torch.equal(fw.weight_grad(delta, ck).double(), want)
    ck = fw.ActCheckpoint(T, d, device=DEV).save(draw(T, d, torch.float32, 6, 2.0 ** 40))
    sums = ck.restore(torch.float32).double().abs().sum(0)
    for e in (-118, -126, -133, -140):
        delta = (draw(T, m, torch.float32, 7).double() * 2.0 ** e).float()
        ref, mag = _wgrad64(delta, ck, 1.0)
        lost = 2.0 ** -133 * sums if m >= 8 else 0 * sums
        assert ((fw.weight_grad(delta, ck).double() - ref).abs() <= (T / 4 + 64) * U * mag + lost).all(), e


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_checkpoint_of_the_largest_numbers(fw, fmt):
    """Nothing saturates: what rounds to the next power of two past a type's
    range restores to an infinity there, as any rounding to fewer bits does."""
    top = torch.finfo(torch.float32).max
    edge = (1.9375 if fmt == "e4m3" else 1.875) * 2.0 ** 127      # half way from the last code to 2^128
    x = torch.full((4, 64), 1.0, device=DEV)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = top, edge, np.nextafter(np.float32(edge), np.float32(0)).item(), -top
    ck = fw.ActCheckpoint(4, 64, fmt, device=DEV).save(x)
    codes, e = A.ckpt_save(f64(x), fmt)
    want = A.ckpt_values(codes, e, 64, fmt)
    assert np.array_equal(ck.codes.cpu().numpy(), codes) and abs(want[[0, 1, 3], 0]).min() == 2.0 ** 128
    with np.errstate(over="ignore"):
        w32 = want.astype(np.float32).astype(np.float64)
    for t in (torch.float32, torch.bfloat16):
        assert np.array_equal(f64(ck.restore(t)), w32)
    assert np.isfinite(w32[2]).all() and np.isposinf(w32[:2, 0]).all() and np.isneginf(w32[3, 0])
    h = torch.full((4, 32), 65504.0, dtype=torch.float16, device=DEV)
    h[1], h[2], h[3] = 63488.0, 61440.0, 61408.0
    ck = fw.ActCheckpoint(4, 32, fmt, device=DEV).save(h)
    assert torch.isinf(ck.restore(torch.float16)[:, 0]).tolist() == [True, True, fmt == "e5m2", False]
    assert ck.restore(torch.float32)[0, 0].item() == 65536.0 and ck.restore()[0, 0].item() == 65536.0
