"""The calls of a served layer together, as a model makes them: the norms around the block, the
heads' norms and rotation with the cache's write, attention with its weights, and eviction when
the cache has reached its budget; and a stack of blocks trained with the norms between them."""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import served as ref
from test_heads import DT, U, f64, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


class Served:
    """One layer of 4 query and 2 key heads, three sequences, a pool of pages handed out by hand."""
    hq, hk, d, page, seqs, width, eps = 4, 2, 64, 8, 3, 6, 1e-6

    def __init__(self, dtype="bf16", kind=torch.int8):
        g = torch.Generator().manual_seed(5)
        dt, cols = DT[dtype], self.hq * self.d

        def new(*s, size=1.0):
            return (size * torch.randn(*s, generator=g)).to(dt).cuda()

        self.w_in = new(cols, (self.hq + 2 * self.hk) * self.d, size=cols ** -0.5)
        self.w_out = new(cols, cols, size=cols ** -0.5)
        self.w_post, self.w_pre, self.wq, self.wk = (1 + new(n, size=0.1) for n in (cols, cols, self.d, self.d))
        self.gate = new(cols)
        self.inv = (10000.0 ** (-torch.arange(self.d // 2) / (self.d // 2))).cuda()
        pages = 2 * self.seqs * self.width
        self.codes = [torch.zeros(pages, self.page, self.hk, self.d, dtype=kind, device="cuda") for _ in range(2)]
        self.scales = [torch.full((pages, self.page, self.hk, 1), float("nan"), device="cuda") for _ in range(2)]
        self.cache = nrm.kv_cache(self.codes[0], self.scales[0], self.codes[1], self.scales[1])
        order = torch.randperm(pages, generator=g).cuda()
        self.tables = order.view(2, self.seqs, self.width).contiguous()
        self.table = self.tables[0].clone()
        self.free = self.tables[1].clone()
        self.lengths = torch.tensor([0, 5, 11], device="cuda")
        self.pos = self.lengths.clone()  # positions in the text, which eviction does not change
        self.weights = torch.zeros(self.seqs, self.hk, self.width * self.page, device="cuda")
        self.stream, self.normed = new(self.seqs, cols), new(self.seqs, cols)
        self.dt = dt
        # what a prompt left: any rows
        n = int(self.lengths.max())
        slots = torch.full((self.seqs, n), -1, device="cuda")
        for s, m in enumerate(self.lengths.tolist()):
            j = torch.arange(m, device="cuda")
            slots[s, :m] = self.table[s, j // self.page] * self.page + j % self.page
        rows = new(self.seqs * n, self.hk, self.d)
        nrm.nrm_kv_cache_write(rows, rows.flip(0).contiguous(), self.cache, slots.flatten())
        qkv = new(self.seqs, self.hq + 2 * self.hk, self.d)
        self.q_out, self.out = torch.empty_like(qkv[:, :self.hq]), torch.empty(self.seqs, self.hq, self.d, dtype=dt, device="cuda")
        self.ws = nrm.kv_attention_workspace(self.out, self.cache, self.table, weights=True)

    def step(self, check):
        qkv = (self.normed @ self.w_in).view(self.seqs, -1, self.d)
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], qkv[:, self.hq + self.hk:]
        slots = self.table.gather(1, (self.lengths // self.page)[:, None])[:, 0] * self.page + self.lengths % self.page
        nrm.nrm_qk_norm_rope_cache(q, k, v, self.wq, self.wk, self.pos, self.inv, self.q_out, None, self.cache, slots, self.eps)
        self.lengths += 1
        self.pos += 1
        before = self.weights.clone()
        nrm.nrm_kv_cache_attention(self.q_out, self.cache, self.table, self.lengths, self.out, self.d ** -0.5, self.ws,
                                   weights=self.weights)
        f = (self.out.view(self.seqs, -1) @ self.w_out)
        x = self.stream.clone()
        nrm.nrm_block_norm_fwd(self.stream, f, self.gate, self.w_post, self.w_pre, self.stream, self.normed, None, None, 0.5, self.eps)
        if not check:
            return
        nrm.nrm_sync_status()
        values = [ref.stored(c.cpu().float().numpy(), s.cpu().numpy(), "int8") for c, s in zip(self.codes, self.scales)]
        want, _, p, _, _ = ref.attention(f64(self.q_out), *values, self.table.cpu().numpy(), self.lengths.cpu().numpy(), self.d ** -0.5)
        # weights rounded to 11 bits and a half step of bfloat16; float32 logits of at most 64 terms
        assert np.abs(f64(self.out) - want).max() <= (2.0 ** -9 + 2.0 ** -10) * max(1.0, np.abs(want).max())
        assert np.abs(f64(self.weights) - f64(before) - p).max() <= 1e-4
        y, _ = ref.block_fwd(f64(x), f64(f), f64(self.gate)[None], f64(self.w_post), 0.5, self.eps)
        assert np.abs(f64(self.stream) - y).max() <= 2.0 ** -8 * np.abs(y).max()
        h, _ = ref.block_pre(f64(self.stream), f64(self.w_pre), self.eps)
        assert np.abs(f64(self.normed) - h).max() <= 2.0 ** -8 * np.abs(h).max()

    def evict(self, keep):
        kept = torch.empty(self.seqs, self.hk, keep, dtype=torch.int64, device="cuda")
        lengths, weights = torch.empty_like(self.lengths), torch.zeros_like(self.weights)
        nrm.nrm_kv_cache_evict(self.cache, self.table, self.lengths, self.weights, self.free, lengths, weights, kept, first=1,
                               recent=4)
        self.table, self.free, self.lengths, self.weights = self.free, self.table, lengths, weights
        return kept


def test_decoding_with_a_budget():
    m = Served()
    for i in range(60):
        m.step(check=i % 7 == 0 or i > 54)
        if int(m.lengths.max()) >= 40:
            weights, lengths = m.weights.cpu().numpy(), m.lengths.cpu().numpy()
            kept = m.evict(20)
            want, new = ref.evict(weights, lengths, 20, 1, 4, weights.shape[2])
            assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(m.lengths.cpu().numpy(), new)
    nrm.nrm_sync_status()
    assert int(m.pos.max()) == 71 and int(m.lengths.max()) < 45


def test_a_step_captured_once_and_replayed():
    # the lengths lie on the device, so one graph serves every step; both against the same steps made one by one
    a, b = Served(), Served()
    b.step(False)
    a.step(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (b.lengths, b.pos)]
    with torch.cuda.graph(graph):
        b.step(False)
    assert all(same(x, y) for x, y in zip(saved, (b.lengths, b.pos)))
    for _ in range(20):
        a.step(False)
        graph.replay()
        assert same(a.stream, b.stream) and same(a.out, b.out) and same(a.weights, b.weights)
    nrm.nrm_sync_status()


def test_training_a_stack_of_blocks():
    # three blocks of a linear layer and SiLU with the norms between them, in float32: gradients of every parameter against
    # those of elementary operations in float64
    rows, cols, blocks, eps, alpha = 40, 96, 3, 1e-5, 0.5
    g = torch.Generator(device="cuda").manual_seed(2)

    def new(*s, size=1.0, mean=0.0):
        return mean + size * torch.randn(*s, generator=g, device="cuda")

    x0 = new(rows, cols)
    W = [new(cols, cols, size=cols ** -0.5) for _ in range(blocks)]
    w_pre, w_post, gates = ([new(*s, size=0.1, mean=1.0) for _ in range(blocks)] for s in ((cols,), (cols,), (4, cols)))
    target = new(rows, cols)
    torch.backends.cuda.matmul.allow_tf32 = False
    # forward: the first norm alone, then a fused call after each block
    r0 = torch.empty(rows, device="cuda")
    h = torch.empty_like(x0)
    nrm.nrm_rmsnorm_fwd(x0, w_pre[0], h, r0, eps)
    x, kept = x0, []
    for i in range(blocks):
        z = h @ W[i]
        f = torch.nn.functional.silu(z)
        last = i + 1 == blocks
        y, nh = torch.empty_like(x), None if last else torch.empty_like(x)
        r1, r2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        nrm.nrm_block_norm_fwd(x, f, gates[i], w_post[i], None if last else w_pre[i + 1], y, nh, r1, r2, alpha, eps)
        kept.append((h, z, f, y, r1, r2))
        x, h = y, nh
    # backward of the loss sum(x * target)
    dy, dh, grads = target, None, {}
    ws = nrm.block_norm_workspace(x0, gates[0])
    for i in reversed(range(blocks)):
        h, z, f, y, r1, r2 = kept[i]
        dx, df, dg, dw = torch.empty_like(x0), torch.empty_like(x0), torch.empty_like(gates[i]), torch.empty_like(w_post[i])
        dwp = None if dh is None else torch.empty_like(w_pre[i])
        nrm.nrm_block_norm_bwd(dh, dy, f, y, gates[i], w_post[i], None if dh is None else w_pre[i + 1], r1, r2, dx, df, dg, dw, dwp, ws,
                               alpha)
        grads["gate", i], grads["post", i] = dg, dw
        if dwp is not None:
            grads["pre", i + 1] = dwp
        s = torch.sigmoid(z)
        dz = df * s * (1 + z * (1 - s))
        grads["W", i] = h.t() @ dz
        dy, dh = dx, dz @ W[i].t()
    first, grads["pre", 0] = torch.empty_like(x0), torch.empty_like(w_pre[0])
    nws = torch.empty(nrm.nrm_workspace_bytes(nrm.NRM_OP_RMSNORM_BWD, rows, cols, nrm.NRM_F32), dtype=torch.uint8, device="cuda")
    nrm.nrm_rmsnorm_bwd(dh, x0, w_pre[0], r0, first, grads["pre", 0], nws)
    grads["x", 0] = first + dy
    nrm.nrm_sync_status()

    p = {("x", 0): x0} | {(n, i): t[i] for n, t in (("W", W), ("pre", w_pre), ("post", w_post), ("gate", gates)) for i in range(blocks)}
    p = {k: t.double().requires_grad_() for k, t in p.items()}

    def norm(t, w):
        return t * ((t * t).mean(-1, keepdim=True) + eps) ** -0.5 * w

    x = p["x", 0]
    for i in range(blocks):
        f = torch.nn.functional.silu(norm(x, p["pre", i]) @ p["W", i])
        x = x + alpha * p["gate", i].repeat_interleave(rows // 4, 0) * norm(f, p["post", i])
    (x * target.double()).sum().backward()
    for key, t in p.items():
        # float32 through three blocks of 96-term products: a few hundred roundings, 2^-24 each, of values of one size
        err = (grads[key].double() - t.grad).norm() / t.grad.norm()
        assert err < 500 * U, (key, float(err))
