"""Block operators where their documentation allows more than an ordinary
cache asks for, each against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import kivi_testlib as T
from test_gpu_blocks import G, Pair, _lib, err, random_list  # noqa: F401  (_lib builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,policy,grp,bits,tiles", [(16384, 0, 4, 2, 700), (16384, 1, 7, 4, 37), (16320, 0, 1, 8, 64),
                                                     (20480, 0, 4, 2, 300), (65440, 0, 2, 2, 20)])
def test_long_windows(R, policy, grp, bits, tiles):
    """The longest tail a window leaves, R + 31 tokens of which 31 values are packed already (or, shared, of whose next
    group 31 tokens are there): more than 256 splits of 64 tokens, and the packed ones beside them."""
    l = R + 31 + G * tiles
    p = Pair(B=2, H=2, T_=l, R=R, policy=policy, grp=grp, bits=bits, lengths=[l, 100], seed=2, capacity=-(-l // R) * R)
    assert p.blocks(0) == tiles
    rng = np.random.default_rng(1)
    lists = np.stack([[random_list(rng, p.blocks(b), 20, "some") for _ in range(2)] for b in range(2)])
    dev, every = torch.from_numpy(lists).cuda(), torch.zeros((2, 2, -(-l // G)), device="cuda")
    for splits in (0, 400):
        p.cache.set_splits(splits)
        every.zero_()
        out = T.out_float(p.cache.attention_blocks(p.q, dev)).reshape(2, 2, grp, 128)
        whole = T.out_float(p.cache.attention_mass(p.q, every)).reshape(2, 2, grp, 128)
        mass = every.cpu().numpy()
        for b in range(2):
            for h in range(2):
                row = lists[b, h][lists[b, h] >= 0].astype(np.int64)
                tokens = np.concatenate([(row[:, None] * G + np.arange(G)).reshape(-1), np.arange(p.blocks(b) * G, p.lengths[b])])
                assert err(out[b, h], p.attend(b, h, tokens)[1], "f16") <= T.ATTN_TOL, (splits, b, h)
                w, ref = p.attend(b, h, np.arange(p.lengths[b]))
                assert err(whole[b, h], ref, "f16") <= T.ATTN_TOL, (splits, b, h)
                per = np.zeros(mass.shape[2])
                np.add.at(per, np.arange(p.lengths[b]) // G, w.sum(0))
                assert np.allclose(mass[b, h], per, rtol=1e-4, atol=1e-6)  # (bounds: test_attention_mass)


@pytest.mark.parametrize("op", ["blocks", "topk", "mass", "mass of long rows"])
def test_an_overlapping_call_reads_what_a_block_operator_wrote(op):
    """The output of a block operator as the queries of an overlapping attention call, and the block operator's own
    queries as that call's output: the last launch that is not an overlapping call has completed by then."""
    from bit_kv_cache_kivi_gb300.kivi import KiviCache
    gen = torch.Generator(device="cuda").manual_seed(5)
    l = 3000 if op == "mass" else 60000

    def make(n):
        c = KiviCache(batch=1, n_kv_heads=2, n_q_heads=8, max_tokens=-(-n // 32) * 32)
        k, v = (torch.randn((1, 2, n, 128), generator=gen, device="cuda", dtype=torch.float16) for _ in range(2))
        c.prefill(k, v)
        return c
    a, b = make(l), make(200)
    b.set_splits(3)  # (the plan does not change with the setting)
    blocks = torch.arange(a.packed_blocks(), dtype=torch.int32, device="cuda").expand(1, 2, -1).contiguous()
    mass = torch.zeros((1, 2, a.cfg.max_tokens // G), device="cuda")
    x, y = (torch.empty((1, 8, 128), dtype=torch.float16, device="cuda") for _ in range(2))

    def run(overlap):
        b.set_overlap(overlap)
        got = []
        for seed in range(20):
            q = torch.randn((1, 8, 128), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").half() * 4
            x.fill_(7.0)
            if op == "blocks":
                a.attention_blocks(q, blocks, out=x)
            elif op == "topk":
                a.attention_topk(q, 1500, out=x)
            else:
                a.attention_mass(q, mass, out=x)
            if not overlap:
                torch.cuda.synchronize()
            b.attention(x, out=y)
            got += [x.clone(), y.clone()]
            # ... and a call that replaces the queries of the one before it
            if op == "blocks":
                a.attention_blocks(q, blocks, out=x)
            elif op == "topk":
                a.attention_topk(q, 1500, out=x)
            else:
                a.attention_mass(q, mass, out=x)
            if not overlap:
                torch.cuda.synchronize()
            b.attention(y, out=q)
            got += [x.clone(), q]
        torch.cuda.synchronize()
        b.set_overlap(False)
        return got
    want = run(False)
    for u, v in zip(want, run(True)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("bits,grp,outliers,qtype", [(2, 4, 0, "f16"), (4, 7, 0, "bf16"), (8, 8, 2, "f32"), (3, 2, 1, "f16"),
                                                     (8, 4, 0, "f16"), (2, 7, 0, "f32")])
def test_entries_that_name_no_block_read_nothing(bits, grp, outliers, qtype):
    """Block 0 full of NaN and infinities, which no list names: holes anywhere in the list, first and last in a warp's share."""
    p = Pair(B=2, H=2, T_=900, bits=bits, grp=grp, outliers=outliers, qtype=qtype, seed=6)
    c, nb = p.cache, p.blocks(0)
    lists = np.full((2, 2, nb), -1, np.int32)
    rng = np.random.default_rng(4)
    for b in range(2):
        for h in range(2):
            at = rng.permutation(nb)[:11]
            lists[b, h, at] = rng.permutation(np.arange(1, nb))[:11]
    lists[1, 0, 1:9] = [nb, 2**31 - 1, -2**31, nb + 7, -1, -1, nb, -1]
    tiles = c.state_views()["tiles"]
    tiles[:, :, 0] = torch.tensor([0x00, 0x7e, 0xff, 0x7f, 0x00, 0x7c, 0x00, 0xfc], dtype=torch.uint8,
                                  device="cuda").repeat(tiles.shape[3] // 8 + 1)[:tiles.shape[3]]
    dev = torch.from_numpy(lists).cuda()
    for splits in (0, 2, 7):
        c.set_splits(splits)
        out = T.out_float(c.attention_blocks(p.q, dev)).reshape(2, 2, grp, 128)
        for b in range(2):
            for h in range(2):
                row = lists[b, h]
                row = row[(row >= 0) & (row < nb)].astype(np.int64)
                tokens = np.concatenate([(row[:, None] * G + np.arange(G)).reshape(-1), np.arange(nb * G, 900)])
                assert err(out[b, h], p.attend(b, h, tokens)[1], qtype) <= T.ATTN_TOL


def test_handles_of_other_shapes_use_one_workspace_in_turn():
    """Their counters lie elsewhere: each zeroes its own when it takes the workspace up again."""
    from bit_kv_cache_kivi_gb300 import kivi
    ps = [Pair(B=1, H=2, T_=3000, seed=1), Pair(B=3, H=2, T_=1400, grp=7, bits=4, seed=2), Pair(B=2, H=2, T_=2000, R=64, seed=3)]
    n = max(max(kivi.kivi_block_workspace_bytes(p.cache.handle), kivi.kivi_attention_workspace_bytes(p.cache.handle)) for p in ps)
    ws = torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
    lists = [torch.arange(p.blocks(0), dtype=torch.int32, device="cuda").expand(p.B, p.H, -1).contiguous() for p in ps]
    want = [(p.cache.attention_blocks(p.q, l), p.cache.attention_mass(p.q, torch.zeros(p.B, p.H, 94, device="cuda")),
             p.cache.attention(p.q)) for p, l in zip(ps, lists)]
    for turn in range(4):
        for p, l, w in zip(ps, lists, want):
            h, rec = p.cache.handle, p.cache._records
            for _ in range(2):
                got = [torch.full_like(p.q, float("nan")) for _ in w]
                kivi.kivi_decode_attention_blocks(h, p.q, kivi.KIVI_F16, l, l.shape[2], got[0], 0.0, ws, n)
                kivi.kivi_decode_attention_mass(h, p.q, kivi.KIVI_F16, got[1], 0.0, None, torch.zeros(p.B, p.H, 94, device="cuda"),
                                                94, 1.0, ws, n, rec, rec.numel())
                assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
                if turn % 2:  # (the whole-cache attention's own layout)
                    kivi.kivi_decode_attention(h, p.q, kivi.KIVI_F16, got[2], 0.0, ws, n)
                    assert torch.equal(got[2], w[2])


def test_a_handle_that_is_gone_leaves_no_trace():
    """Handles come and go beside one that keeps its workspace."""
    p = Pair(T_=1000)
    blocks = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, 2, 20).contiguous()
    want = p.cache.attention_blocks(p.q, blocks)
    others = [Pair(T_=300 + 50 * i) for i in range(4)]
    for i in (1, 3, 0, 2):
        others[i].cache.attention_blocks(others[i].q, blocks)
        others[i] = None
        assert torch.equal(p.cache.attention_blocks(p.q, blocks), want)


# f32 outputs are 3e-6 of a head's largest output off, 5e-6 at 8 bits, 1e-5 over 131k tokens (the figures that the block
# attention is documented with).  Of the 1000 tokens here four times the first stays below what is lost where a weight
# is one fp16 number: a rounding of up to 2^-11 a weight, 2^-11 / sqrt(12) = 1.4e-4 on the average of many, and as much of
# an output that is their mean.  The second assertion holds the bound to that, with the rounding put into the formula.
F32_TOL = 2e-5


@pytest.mark.parametrize("bits,policy,R,grp,outliers", [
    (2, 0, 32, 4, 0), (2, 0, 64, 7, 0), (3, 1, 32, 3, 0), (3, 0, 32, 8, 1), (4, 0, 96, 8, 0), (4, 1, 128, 1, 0),
    (8, 0, 32, 4, 0), (8, 1, 64, 7, 0), (8, 0, 128, 8, 2), (2, 0, 256, 5, 0), (8, 0, 32, 1, 4), (4, 0, 32, 18, 0)])
def test_f32_outputs_tell_a_pair_from_one_weight(bits, policy, R, grp, outliers):
    p = Pair(T_=1000, R=R, bits=bits, policy=policy, grp=grp, qtype="f32", lengths=[1000, 871], outliers=outliers, seed=9)
    rng = np.random.default_rng(2)
    lists = np.stack([[random_list(rng, p.blocks(b), 15, "some") for _ in range(2)] for b in range(2)])
    for splits in (0, 3, 9):
        p.cache.set_splits(splits)
        out = p.cache.attention_blocks(p.q, torch.from_numpy(lists).cuda()).cpu().numpy().reshape(2, 2, grp, 128)
        whole = p.cache.attention_mass(p.q, torch.zeros((2, 2, 32), device="cuda")).cpu().numpy().reshape(2, 2, grp, 128)
        for b in range(2):
            for h in range(2):
                row = lists[b, h][lists[b, h] >= 0].astype(np.int64)
                tokens = np.concatenate([(row[:, None] * G + np.arange(G)).reshape(-1), np.arange(p.blocks(b) * G, p.lengths[b])])
                for got, at in ((out, tokens), (whole, np.arange(p.lengths[b]))):
                    w, ref = p.attend(b, h, at)
                    assert T.attn_err(got[b, h], ref) <= F32_TOL, (splits, b, h)
                    one = (w / w.max(1, keepdims=True)).astype(np.float16).astype(np.float64)
                    lost = (one / one.sum(1, keepdims=True)) @ p.kv(b, h)[1][at]
                    assert T.attn_err(lost, ref) > 2 * F32_TOL


@pytest.mark.parametrize("B,H,grp,bits,n,one", [(152, 8, 4, 2, 8, True), (87, 7, 4, 2, 8, False), (64, 8, 2, 8, 5, True),
                                                (86, 8, 7, 4, 9, True), (1500, 1, 1, 3, 1, True)])
def test_short_lists_of_very_many_units(B, H, grp, bits, n, one):
    """More units than CTAs run at once: list and window in one CTA a unit, which writes no partials, from one and a half
    rounds of them on."""
    from bit_kv_cache_kivi_gb300 import kivi
    T_ = 330
    p = Pair(B=2, H=H, T_=T_, bits=bits, grp=grp, lengths=[T_, 41], seed=n)
    lists = np.stack([[random_list(np.random.default_rng(h), p.blocks(b), n, "some") for h in range(H)] for b in range(2)])
    c = kivi.KiviCache(batch=B, n_kv_heads=H, n_q_heads=H * grp, max_tokens=352, bits=bits)
    rep = lambda x: x.repeat(B // 2 + 1, *[1] * (x.dim() - 1))[:B].contiguous()  # noqa: E731
    c.prefill(rep(T.dev(p.wl.k, "f16")), rep(T.dev(p.wl.v, "f16")), ([T_, 41] * B)[:B] if B <= 1024 else None)
    size = kivi.kivi_block_workspace_bytes(c.handle)
    ws = torch.full((size,), 0x55, dtype=torch.uint8, device="cuda")
    q, out = rep(p.q), torch.full((B, H * grp, 128), float("nan"), device="cuda", dtype=torch.float16)
    kivi.kivi_decode_attention_blocks(c.handle, q, kivi.KIVI_F16, rep(torch.from_numpy(lists).cuda()), n, out, 0.0, ws, size)
    if B <= 1024:  # (else the two sequences are of one length, and differ from p's second)
        assert torch.equal(out, rep(out[:2]))
    got = T.out_float(out[:2].contiguous()).reshape(2, H, grp, 128)
    for b in range(2 if B <= 1024 else 1):
        for h in range(H):
            row = lists[b, h][lists[b, h] >= 0].astype(np.int64)
            tokens = np.concatenate([(row[:, None] * G + np.arange(G)).reshape(-1), np.arange(p.blocks(b) * G, p.lengths[b])])
            assert err(got[b, h], p.attend(b, h, tokens)[1], "f16") <= T.ATTN_TOL
    partials = B * H * 8 * 128 * 4  # the first split's outputs of every unit, and more behind them
    assert bool((ws[:partials] == 0x55).all()) == one


# ------------------------------------------------------------------ long rows, many units

@pytest.mark.parametrize("B,H,grp,bits,blocks,outliers,qtype", [
    (16, 4, 4, 2, 1000, 0, "f16"), (16, 4, 7, 4, 1000, 0, "bf16"), (8, 8, 18, 8, 1000, 0, "f32"), (16, 4, 9, 3, 515, 2, "f16"),
    (1, 8, 4, 2, 6001, 0, "f16"), (16, 40, 3, 2, 130, 1, "f16")])
def test_scores_of_many_groups(B, H, grp, bits, blocks, outliers, qtype):
    """Rows of more groups of 64 blocks than CTAs share them: tables of q used again for the next group, or made again
    where the heads take several rounds."""
    from bit_kv_cache_kivi_gb300.kivi import KiviCache, key_scale_pos
    l, L = blocks * G + 32 + 9, 2 ** bits - 1
    gen = torch.Generator(device="cuda").manual_seed(blocks + grp)
    c = KiviCache(batch=B, n_kv_heads=H, n_q_heads=H * grp, max_tokens=-(-l // 32) * 32, bits=bits, outliers=outliers)
    lengths = [l] + [int(x) for x in np.random.default_rng(1).integers(l // 3, l, B - 1)]
    k = torch.randn((B, H, l, 128), generator=gen, device="cuda", dtype=torch.float16)
    k[:, :, :, 5] *= 4
    c.prefill(k, k, lengths)
    q = torch.randn((B, H * grp, 128), generator=gen, device="cuda").to({"f16": torch.float16, "bf16": torch.bfloat16,
                                                                        "f32": torch.float32}[qtype])
    del k
    n = blocks + 70
    out = torch.full((B, H, n), float("nan"), device="cuda")
    c.block_scores(q, out=out)
    lv = c.layout_views()
    at = torch.tensor([key_scale_pos(ch, bits) for ch in range(128)], device="cuda")
    ref = torch.full((B, H, blocks), -float("inf"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref)
    for b in range(B):
        nb = c.packed_blocks(b)
        z, s = (lv[x][b, :, :nb, at].view(torch.float16).double() for x in ("zero_k", "scale_k"))
        qb = q[b].double().view(H, grp, 128)
        qmax = qb.abs().amax(2)
        for j in range(grp):
            x = qb[:, j, None, :]
            value = torch.maximum(x * z, x * (z + L * s)).sum(2)
            size = ((x * z).abs() + L * (x * s).abs()).sum(2)
            if outliers:
                idx = lv["outl_idx"][b, :, :nb, :outliers].long()
                val = lv["outl_val"][b, :, :nb].contiguous().view(torch.float16).double()
                prod = torch.gather(x.expand(H, nb, 128), 2, idx)[:, :, None] * val
                value += prod.sum(3).amax(2)
                size += prod.abs().sum(3).amax(2)
            ref[b, :, :nb] = torch.maximum(ref[b, :, :nb], value)
            # (the bound of test_scores)
            t = (2.0 ** -16 + 2.0 ** -22) * size + 2.0 ** -24 * qmax[:, j, None] * size.amax(1, keepdim=True)
            tol[b, :, :nb] = torch.maximum(tol[b, :, :nb], t)
        assert torch.all(out[b, :, nb:] == -float("inf"))
        assert torch.all((out[b, :, :nb].double() - ref[b, :, :nb]).abs() <= tol[b, :, :nb])


@pytest.mark.parametrize("place", ["in place", "into", "into, over the masses"])
@pytest.mark.parametrize("bits,policy,R,outliers,blocks,keep,first,last,kind", [
    (2, 0, 32, 0, 513, 200, 1, 2, "normal"), (3, 1, 64, 2, 600, 599, 0, 0, "ties"), (4, 0, 128, 0, 1100, 37, 4, 8, "ties"),
    (8, 1, 32, 0, 1025, 1000, 0, 9, "odd"), (2, 0, 64, 4, 4200, 2100, 2, 3, "normal"), (2, 0, 32, 0, 4097, 4095, 0, 0, "equal"),
    (4, 0, 32, 0, 4096, 0, 0, 0, "narrow")])
def test_evictions_of_long_rows(place, bits, policy, R, outliers, blocks, keep, first, last, kind):
    """Past the rows that one launch evicts: every selection of more than 512 blocks, and the copies behind it."""
    from bit_kv_cache_kivi_gb300.kivi import KiviCache
    from test_gpu_blocks import live_tiles, rough, select_ref
    B, H = 3, 2
    lengths = [blocks * G + R + 7, (blocks * 2 // 3) * G + R, 5]
    new_cache = lambda n: KiviCache(batch=B, n_kv_heads=H, n_q_heads=H, max_tokens=-(-n // R) * R, bits=bits, residual=R,  # noqa: E731
                                    policy=policy, outliers=outliers)
    c = new_cache(max(lengths))
    gen = torch.Generator(device="cuda").manual_seed(keep)
    for x in c.buffers.values():
        x.copy_(torch.randint(0, 256, x.shape, generator=gen, device="cuda", dtype=torch.uint8))
    c.set_lengths(lengths)
    before = {n: x.clone() for n, x in c.state_views().items()}
    nb, left = [c.packed_blocks(b) for b in range(B)], [c.evict_left(keep, b) for b in range(B)]
    assert nb[0] == blocks
    new = [lengths[b] - G * (nb[b] - left[b]) for b in range(B)]
    row = -(-max(lengths) // G) + 1
    mn = rough(np.random.default_rng(blocks), (B, H, row), kind)
    mass = torch.from_numpy(mn).cuda()
    out_row, to = row, c
    if place != "in place":
        to = new_cache(max(new))
        to.buffers["tiles"].fill_(0xA5)
    if place == "into":
        out_row = -(-max(new) // G) + 1
        mass_out = torch.full((B, H, out_row), float("nan"), device="cuda")
    else:
        mass_out = mass
    kept = c.evict_blocks(mass, keep, keep_first=first, keep_last=last, into=None if to is c else to, mass_out=mass_out)
    kn, mo, after = kept.cpu().numpy(), mass_out.cpu().numpy(), to.state_views()
    assert to.lengths == new and kn.shape == (B, H, max(left))
    if to is not c:
        assert c.lengths == lengths and all(torch.equal(c.state_views()[n], before[n]) for n in before)
    for b in range(B):
        tail = live_tiles(lengths[b], R, policy) - nb[b]
        held = -(-lengths[b] // G) - nb[b]
        for h in range(H):
            want = select_ref(mn[b, h], nb[b], left[b], first, last)[:left[b]]
            assert np.array_equal(kn[b, h], np.concatenate([want, np.full(max(left) - left[b], -1)]))
            src = np.concatenate([want, np.arange(nb[b], nb[b] + tail)]).astype(int)
            assert torch.equal(after["tiles"][b, h, :len(src)], before["tiles"][b, h][torch.from_numpy(src).cuda()])
            if to is not c:
                assert torch.all(after["tiles"][b, h, len(src):] == 0xA5)
            elif left[b] < nb[b]:
                assert torch.equal(after["tiles"][b, h, nb[b] + tail:], before["tiles"][b, h, nb[b] + tail:])
            for ring in ("ring_k", "ring_v"):
                assert torch.equal(after[ring][b, h], before[ring][b, h])
            m = np.concatenate([mn[b, h][want], mn[b, h][nb[b]:nb[b] + held]])
            assert np.array_equal(mo[b, h], np.concatenate([m, np.zeros(out_row - len(m), np.float32)]), equal_nan=True)


def test_captured_with_overlapping_calls():
    """Block operators and overlapping attention calls that read what they wrote, in one graph and replayed."""
    a, b = Pair(B=1, H=2, T_=20000, grp=4, seed=1), Pair(B=1, H=2, T_=200, grp=4, seed=2)
    blocks = torch.arange(a.blocks(0), dtype=torch.int32, device="cuda").expand(1, 2, -1).contiguous()
    mass, new = torch.rand((1, 2, 640), device="cuda"), torch.empty((1, 2, 640), device="cuda")
    q = a.q.clone()
    outs = [torch.empty_like(q) for _ in range(7)]
    b.cache.set_splits(3)  # (the plan does not change with the setting)

    def calls(x, overlap):
        b.cache.set_overlap(overlap)
        a.cache.attention_blocks(q, blocks, out=x[0])
        b.cache.attention(x[0], out=x[1])
        b.cache.attention(x[0], out=x[2])
        a.cache.attention_mass(x[1], mass, mass_out=new, out=x[3])
        b.cache.attention(x[3], out=x[4])
        a.cache.attention_topk(x[4], 400, out=x[5])
        b.cache.attention(x[5], out=x[6])
        b.cache.set_overlap(False)
    calls(outs, False)  # (the scratch is made by the first calls)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(outs, True)
    for seed in range(6):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).half() * 4)
        for x in outs:
            x.fill_(7.0)
        g.replay()
        got = [x.clone() for x in outs + [new]]
        want = [torch.empty_like(q) for _ in outs]
        calls(want, False)
        assert all(torch.equal(x, y) for x, y in zip(got, want + [new]))


@pytest.mark.parametrize("grp,outliers", [(4, 0), (9, 2)])
def test_scores_of_nan(grp, outliers):
    """A head whose q holds a NaN counts for no block, a block whose scales hold one for no head."""
    p = Pair(B=2, H=2, T_=400, grp=grp, outliers=outliers, qtype="f32", seed=3)
    c, nb = p.cache, p.blocks(0)
    q = p.q.clone()
    first = c.block_scores(q, out=torch.empty((2, 2, nb), device="cuda"))
    heads = q.view(2, 2, grp, 128)
    heads[0, 0, 1, 17] = float("nan")
    rest = heads.clone()
    rest[0, 0, 1] = rest[0, 0, 0]  # (a head twice changes no maximum)
    got = c.block_scores(q, out=torch.empty_like(first))
    assert torch.equal(got, c.block_scores(rest.view(q.shape), out=torch.empty_like(first)))
    heads[1, 1] = float("nan")
    got = c.block_scores(q, out=torch.empty_like(first))
    assert torch.all(got[1, 1] == -float("inf")) and torch.equal(got[1, 0], first[1, 0])
    c.layout_views()["scale_k"][0, 1, 3, 40] = 0x7e00
    got = c.block_scores(p.q, out=torch.empty_like(first))
    assert got[0, 1, 3] == -float("inf")
    keep = torch.ones_like(first, dtype=torch.bool)
    keep[0, 1, 3] = False
    assert torch.equal(got[keep], first[keep])


@pytest.mark.parametrize("bits,policy,R,grp,outliers", [(2, 0, 32, 4, 0), (4, 0, 128, 7, 0), (8, 1, 64, 4, 2), (3, 1, 32, 8, 0),
                                                       (2, 0, 96, 18, 1)])
def test_memory_behind_the_tokens_counts_for_nothing(bits, policy, R, grp, outliers):
    """The cache's unused tiles and ring slots, scratch, records and outputs full of NaN or of zeros: the same results."""
    from bit_kv_cache_kivi_gb300 import kivi
    lengths = [611, 1, R + 31, 2 * R + 33]
    wl = Pair(B=4, H=2, T_=611, R=R, bits=bits, policy=policy, grp=grp, outliers=outliers, lengths=lengths, seed=8).wl
    got = []
    for byte in (0x00, 0x7f, 0xff):
        c = T.gpu_cache(wl, capacity=R * -(-704 // R), policy=policy, outliers=outliers)
        for x in c.buffers.values():
            x.fill_(byte)
        c.prefill(T.dev(wl.k, "f16"), T.dev(wl.v, "f16"), lengths)
        q = T.dev(wl.q, "f16")
        rows = lambda n, dtype=torch.float32: torch.full((4, 2, 4 * n), byte, dtype=torch.uint8, device="cuda").view(dtype)  # noqa: E731
        nws, nrec = kivi.kivi_block_workspace_bytes(c.handle), kivi.kivi_block_records_bytes(c.handle)
        ws, rec = (torch.full((n,), byte, dtype=torch.uint8, device="cuda") for n in (nws, nrec))
        scores, blocks, mass = rows(25), rows(6, torch.int32), rows(25)
        o1, o2, o3 = (torch.full((q.numel() * 2,), byte, dtype=torch.uint8, device="cuda").view(torch.float16).view(q.shape) for _ in range(3))
        h = c.handle
        kivi.kivi_decode_attention_topk(h, q, kivi.KIVI_F16, 6, 1, 1, scores, 25, blocks, o1, 0.0, ws, nws)
        lists = torch.tensor([3, 0, -1, 9, 2, 2], dtype=torch.int32, device="cuda").expand(4, 2, 6).contiguous()
        kivi.kivi_decode_attention_blocks(h, q, kivi.KIVI_F16, lists, 6, o2, 0.0, ws, nws)
        kivi.kivi_decode_attention_mass(h, q, kivi.KIVI_F16, o3, 0.0, None, mass, 25, 1.0, ws, nws, rec, nrec)
        kept, left = rows(25, torch.int32), rows(25)
        c.evict_blocks(mass, 3, kept=kept, mass_out=left)
        got.append([scores, blocks, o1, o2, o3, mass, kept, left, c.attention(q)])
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    assert all(bool(torch.isfinite(x).all()) for x in got[0][2:])
