"""Kernels that are launched while their predecessor in the stream still runs, and wait for its end
on the device: what they read after the wait must not go through the read-only path, which wants
memory that nobody writes while the kernel lives.  The sources are checked for it without a GPU; on
one, calls that read what the call before them wrote are compared with the same calls one at a time."""
import os
import re

import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from normalization_layernorm_rmsnorm_gb300 import build as nbuild


def code(name):
    """A source file without its comments."""
    text = open(os.path.join(nbuild.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """(signature, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.start())
        depth, i = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        yield text[m.start():start], text[start:i]


@pytest.mark.parametrize("name", ["heads.cuh", "rownorm.cuh"])
def test_waiting_kernels_do_not_use_the_read_only_path(name):
    found = 0
    for signature, body in kernels(code(name)):
        if "pdl_wait()" in body or "pdl_next()" in body:
            found += 1
            bad = [word for word in ("__restrict__", "__ldg", ".nc") if word in signature + body]
            assert not bad, signature
    assert found


def test_kernels_on_heads_have_no_read_only_loads():
    # every kernel of the file waits for its predecessor, and so does all that their helpers read
    text = code("heads.cuh")
    for signature, body in kernels(text):
        assert "pdl_next()" in body, signature
    # (the named helpers of common.cuh load through it)
    assert re.findall(r"__ldg|\.nc\b|__restrict__|ld_stream_v4|ld_cached_v4|load_vec", text) == []


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_chain_of_calls_reads_what_the_call_before_wrote(captured):
    # each call's output is the next one's rows, weights, frequencies, codes or scales, with no other
    # kernel between them, in buffers that are written anew each time
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tokens, heads, d = 4000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(3)

    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, device="cuda", dtype=dtype)

    src, dy, w0 = new(tokens, heads, d), new(tokens, heads, d), torch.ones(d, device="cuda", dtype=torch.bfloat16)
    rstd, freq_src, zero = new(tokens * heads, dtype=torch.float32), new(1, 1, d // 2, dtype=torch.float32), torch.zeros(
        1, dtype=torch.int64, device="cuda")
    quiet = torch.zeros(1, device="cuda")  # a frequency of 0: the rotation copies
    wsrc = new(1, 1, d)
    pos, slots = torch.arange(tokens, device="cuda"), torch.randperm(tokens, generator=g, device="cuda")
    codes = [new(tokens // 8, 8, heads, d, dtype=torch.int8) for _ in range(2)]
    scales = [new(tokens // 8, 8, heads, 2, dtype=torch.float32) for _ in range(2)]
    cache = nrm.kv_cache(codes[0], scales[0], codes[1], scales[1])
    o = dict(dx=new(tokens, heads, d), w=new(1, 1, d), freq=new(1, 1, d // 2, dtype=torch.float32), q=new(tokens, heads, d),
             k=new(tokens, heads, d), rq=new(tokens, heads, dtype=torch.float32), rk=new(tokens, heads, dtype=torch.float32),
             kb=new(tokens, heads, d), vb=new(tokens, heads, d), dq=new(tokens, heads, d), dk=new(tokens, heads, d), dwq=new(d),
             dwk=new(d), k2=new(tokens, heads, d), v2=new(tokens, heads, d))
    ws = nrm.qk_norm_workspace(src)
    between = [lambda: None]

    def chain():
        step = between[0]
        # (its main kernel lets its successor be launched before its last stores)
        nrm.nrm_rmsnorm_bwd(dy.view(-1, d), src.view(-1, d), w0, rstd, o["dx"].view(-1, d), None, None), step()
        nrm.nrm_rope_fwd(wsrc, None, zero, quiet, o["w"], None), step()
        nrm.nrm_rope_fwd(freq_src, None, zero, quiet, o["freq"], None), step()
        w, freq = o["w"].view(d), o["freq"].view(d // 2)
        nrm.nrm_qk_norm_rope_fwd(o["dx"], src, w, w, pos, freq, o["q"], o["k"], o["rq"], o["rk"], 1e-6), step()
        nrm.nrm_kv_cache_write(o["k"], o["q"], cache, slots), step()
        nrm.nrm_kv_cache_read(cache, slots, o["kb"], o["vb"]), step()
        nrm.nrm_rope_fwd(wsrc, None, zero, quiet, o["w"], None), step()
        nrm.nrm_qk_norm_rope_bwd(o["kb"], o["vb"], o["dx"], src, w, w, o["rq"], o["rk"], pos, freq, o["dq"], o["dk"], o["dwq"],
                                 o["dwk"], ws), step()
        nrm.nrm_qk_norm_rope_cache(o["dq"], o["dk"], o["vb"], o["dwq"], o["dwk"], pos, freq, o["q"], None, cache, slots,
                                   1e-6), step()
        nrm.nrm_kv_cache_read(cache, slots, o["k2"], o["v2"]), step()

    def refresh():
        for t in (src, dy, wsrc):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g).bfloat16())
        rstd.copy_(torch.rand(rstd.shape, device="cuda", generator=g) + 0.5)
        freq_src.copy_(torch.rand(freq_src.shape, device="cuda", generator=g))
        torch.cuda.synchronize()

    refresh()
    graph = torch.cuda.CUDAGraph()
    if captured:
        chain()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            chain()
    for i in range(30):
        refresh()
        graph.replay() if captured else chain()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in o.items()}
        for t in (*o.values(), *codes, *scales):
            t.zero_()
        torch.cuda.synchronize()
        between[0] = torch.cuda.synchronize
        chain()
        between[0] = lambda: None
        for n, t in o.items():
            assert torch.equal(t.view(torch.uint8), got[n].view(torch.uint8)), (i, n)
    nrm.nrm_sync_status()
