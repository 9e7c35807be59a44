"""Linear attention and the layer norm where offsets pass 32 bits: the same numbers at far strides, heads and slots give the
bits that they give side by side (64-bit forms are compared in test_linattn_gpu.py and test_layernorm_gpu.py)."""
import pytest
import torch

from bidirectional_selective_scan_amd import attention, binding, block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rnd(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def run_all(q, k, v, g):
    fwd = binding.PreparedLinAttn(q, k, v, g)
    y = fwd()
    grad = binding.PreparedLinAttnGrad(fwd, dy=rnd(*v.shape, seed=9))
    grad()
    return [t.clone() for t in (y, fwd.h_last, grad.dq, grad.dk, grad.dv, grad.dlog_decay)]


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_rows_past_32_bits():
    # 600 rows (cut into segments), each as far apart as rows may be: 5 GB from the first to the last
    T, H, dk, dv, ld = 600, 2, 16, 24, (1 << 22) - 8
    q, k, v = rnd(1, T, H, dk, seed=1), rnd(1, T, H, dk, seed=2), rnd(1, T, H, dv, seed=3)
    g = -rnd(1, T, H, seed=4, dtype=torch.float32).abs()
    big = torch.empty(T, ld, dtype=torch.bfloat16, device=DEV)
    assert big.numel() > 1 << 31
    at, far = 0, []
    for t in (q, k, v):
        n = t.shape[2] * t.shape[3]
        big[:, at:at + n] = t.view(T, n)
        far.append(big[:, at:at + n].view(1, T, *t.shape[2:]))
        at += n
    assert binding.PreparedLinAttn(*far, g).plan["chunks"] > 1
    same(run_all(*far, g), run_all(q, k, v, g))
    x, w, b = rnd(T, 768, seed=5), rnd(768, seed=6, dtype=torch.float32), rnd(768, seed=7, dtype=torch.float32)
    big[:, 4096:4096 + 768] = x
    same([block.layer_norm(big[:, 4096:4096 + 768], weight=w, bias=b)[1]], [block.layer_norm(x, weight=w, bias=b)[1]])


def test_heads_past_32_bits():
    T, H, d = 70, 2, 16
    q, k, v = (rnd(1, T, H, d, seed=s) for s in (1, 2, 3))
    g = -rnd(1, T, H, seed=4, dtype=torch.float32).abs()
    far = (1 << 31) + 64
    big = torch.empty(far + 3 * T * d, dtype=torch.bfloat16, device=DEV)
    views = []
    for n, t in enumerate((q, k, v)):
        w = torch.as_strided(big, (1, T, H, d), (T * d, d, far, 1), n * T * d)
        w.copy_(t)
        views.append(w)
    same(run_all(*views, g), run_all(q, k, v, g))


def test_slots_past_32_bits():
    B, H, d = 3, 24, 64
    slots = (1 << 31) // (H * d * d) + 4
    q, k, v = (rnd(B, H, d, seed=s) for s in (1, 2, 3))
    g = -rnd(H, seed=4, dtype=torch.float32).abs()
    state = torch.empty(slots, H, d, d, device=DEV)
    near = rnd(B, H, d, d, seed=5, dtype=torch.float32)
    at = [slots - 1, 0, slots - 3]
    for b, s in enumerate(at):
        state[s] = near[b]
    y = attention.linattn_step(q, k, v, g, state, slots_in=torch.tensor(at, dtype=torch.int32, device=DEV))
    want = attention.linattn_step(q, k, v, g, near)
    same([y] + [state[s] for s in at], [want] + list(near))
