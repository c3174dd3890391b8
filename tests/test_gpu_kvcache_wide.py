"""The paged cache where its arrays are large: offsets past 32 bits, an append captured once and replayed at other lengths, and
more sequences than a grid's dimension holds.  Equal bit for bit to the float64 definition, K and V, codes and exponents."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_34_gb300 import specverify as sv
from tests.test_gpu_kvcache import Pair, dev, values

pytestmark = pytest.mark.gpu


def test_replayed_appends_past_4_gib():
    H, page, D, n = 8, 128, 128, 5
    P = (1 << 32) // (H * page * D) + 3
    ref = Pair(6, 1, H, page, D, 3, spare=0)
    ref.table = np.array([[2, 0, 1]], np.int32)
    cache = sv.alloc_kv_cache(P, H, page, D)
    for mine, known in zip(cache.tensors, ref.gpu.tensors):
        mine[P - 3:] = known                                # the last three pages hold what the definition's do
    table = dev(ref.table + (P - 3))
    k, v = (torch.zeros(1, n, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    length, num = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fn = sv.prepare_kv_append(k, v, cache, table, length, num, st)
        fn()                                                # (no token)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fn()
    rng = np.random.default_rng(7)
    for at, m in ((0, 5), (130, 5), (254, 5), (3, 1), (126, 4), (200, 0), (379, 5)):
        x, y = (values(rng, (1, n, H, D), torch.bfloat16) for _ in range(2))
        k.copy_(x), v.copy_(y), length.fill_(at), num.fill_(m)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert ref.host.append(ref.table[0], at, x[0, :m].double().numpy(), y[0, :m].double().numpy()) == 0
        for w, (c, e) in enumerate(((cache.k_codes, cache.k_exp), (cache.v_codes, cache.v_exp))):
            assert np.array_equal(e[P - 3:].cpu().numpy(), ref.host.exps[w]), (at, w)
            assert np.array_equal(c[P - 3:].cpu().numpy(), ref.host.codes[w]), (at, w)
        out = [torch.full((1, n, H, D), 5.5, device="cuda") for _ in range(2)]
        sv.spec_kv_read(cache, table, length, num, *out, st)
        torch.cuda.synchronize()
        for got, want in zip(out, ref.host.read(ref.table[0], at, m)):
            assert (got[0, m:] == 5.5).all()
            if m:
                assert np.array_equal(got[0, :m].double().cpu().numpy(), np.stack(want))
    assert int(st) == 0


def test_more_sequences_than_a_grid_dimension():
    B, n, H, page, D = 65535 + 400, 3, 1, 16, 64
    p = Pair(8, B, H, page, D, 1)
    look = [0, 1, 777, 65533, 65534, 65535, 65536, 65537, B - 2, B - 1]
    rng = np.random.default_rng(9)
    first = rng.integers(0, 14, B).astype(np.int32)
    num = rng.integers(0, n + 1, B).astype(np.int32)
    num[look] = n
    first[65535], num[65534] = -1, 9
    k, v = (torch.randn(B, n, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    table, firsts = dev(p.table), dev(first)
    want = np.zeros(B, int)
    want[65534], want[65535] = sv.ST_CLAMPED_GAMMA, sv.ST_BAD_PAGE

    def same():
        torch.cuda.synchronize()
        for b in look:
            page_of = int(p.table[b, 0])
            for w, (c, e) in enumerate(((p.gpu.k_codes, p.gpu.k_exp), (p.gpu.v_codes, p.gpu.v_exp))):
                assert np.array_equal(e[page_of].cpu().numpy(), p.host.exps[w][page_of]), (b, w)
                assert np.array_equal(c[page_of].cpu().numpy(), p.host.codes[w][page_of]), (b, w)

    sv.spec_kv_append(k, v, p.gpu, table, firsts, dev(num), st)
    for b in look:
        p.host.append(p.table[b], int(first[b]), k[b].double().cpu().numpy(), v[b].double().cpu().numpy())
    same()
    assert np.array_equal(st.cpu().numpy(), want)
    st.zero_()
    out = [torch.full((B, n, H, D), 5.5, device="cuda") for _ in range(2)]
    sv.spec_kv_read(p.gpu, table, firsts, dev(num), *out, st)
    torch.cuda.synchronize()
    assert np.array_equal(st.cpu().numpy(), want)
    for b in look:
        for got, x in zip(out, p.host.read(p.table[b], int(first[b]), n)):
            for i in range(n):
                assert np.array_equal(got[b, i].double().cpu().numpy(), np.full((H, D), 5.5) if first[b] < 0 else x[i]), (b, i)
    # node 2 of each tree of two follows the root (the block begins below position 13)
    st.zero_()
    base = np.where(first < 0, first, np.minimum(first, 12)).astype(np.int32)
    path = torch.tensor([2, -1], dtype=torch.int32, device="cuda").repeat(B, 1)
    accepted = torch.ones(B, dtype=torch.int32, device="cuda")
    sv.spec_kv_keep_path(p.gpu, table, dev(base), path, accepted, status=st)
    for b in look:
        p.host.keep_path(p.table[b], int(base[b]), [2], True, 2)
    same()
    want[65534] = 0
    assert np.array_equal(st.cpu().numpy(), want)
