"""The paged-cache attention operators on the GPU against plain fp64 references."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp

pytestmark = pytest.mark.gpu


def on_device(c, attn):
    if c["kv"] != "bf16":
        attn.set_scales(c["ks"].cuda(), c["vs"].cuda())
    return tp.PagedCache(attn, c["K"].cuda(), c["V"].cuda(), c["table"].cuda(), c["lens"].cuda())


def ok(attn):
    torch.cuda.synchronize()
    rc, detail = attn.status()
    assert rc == tp.TPMLP_OK, f"device status {rc} ({detail:#x})"


def queries(rows, Hq, D, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    return torch.randn((rows, Hq * D), generator=g).bfloat16()


def check_rows(c, q, got, lse, spans, Hq, D, scale):
    """spans: (row, sequence, lo, hi) of every row that must have been written."""
    out, lse = got.cpu().double().view(-1, Hq, D), lse.cpu().double()
    for r, b, lo, hi in spans:
        o, l, spread, big = ref.attend(c, b, q[r].double().view(Hq, D), hi, lo, scale)
        tol = ref.out_tolerance(o, spread, c["kv"])
        err = (out[r] - o).abs()
        assert bool((err <= tol).all()), (r, b, lo, hi, float((err / tol).max()))
        if hi <= lo:
            assert bool((lse[r] == -math.inf).all())
        else:
            assert bool(((lse[r] - l).abs() <= ref.lse_tolerance(l, big, D)).all()), (r, b, lo, hi)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved,T", [
    (4, 4, 128, 16, 128, False, 1),
    (12, 2, 64, 32, 64, True, 37),
    (5, 5, 64, 16, 32, False, 130),
    (24, 3, 128, 64, 48, True, 65),
    (16, 1, 128, 256, 96, False, 9),
    (3, 1, 64, 128, 0, False, 7),
])
def test_append_matches_definition(lib, kv, Hq, Hkv, D, page, rot, interleaved, T):
    lens = [200, 1, 77]
    c = ref.make(Hkv, D, page, kv, lens, seed=T)
    g = torch.Generator().manual_seed(T)
    width = (Hq + 2 * Hkv) * D
    qkv = torch.randn((T, width + 8), generator=g).bfloat16()  # rows wider than the three parts
    # distinct (sequence, position) places, some tokens skipped
    places = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    pick = torch.randperm(len(places), generator=g)[:T].tolist()
    seq = torch.tensor([places[i][0] for i in pick], dtype=torch.int32)
    pos = torch.tensor([places[i][1] for i in pick], dtype=torch.int32)
    pos[::5] = -1 if T > 5 else pos[::5]
    freq = [1e4 ** (-2 * i / rot) for i in range(rot // 2)] if rot else []
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        if rot:
            attn.set_rope(rot, interleaved=interleaved)
        cache = on_device(c, attn)
        d = qkv.cuda()
        q, k, v = d[:, :Hq * D], d[:, Hq * D:(Hq + Hkv) * D], d[:, (Hq + Hkv) * D:width]
        q_out = torch.full((T, Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
        attn.append(q, k, v, cache, pos.cuda(), seq.cuda(), q_out=q_out)
        ok(attn)
        inplace = attn.append(q, k, v, cache, pos.cuda(), seq.cuda(), q_out=q)
        ok(attn)
        kept = pos >= 0
        assert torch.equal(inplace[kept], q_out[kept])
        assert bool((q_out[~kept] == 7.0).all())  # skipped tokens are not written
        K, V = cache.K.cpu().float().double(), cache.V.cpu().float().double()
    x = qkv.double()
    wantq = x[:, :Hq * D].view(T, Hq, D)
    wantk = x[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D)
    wantv = x[:, (Hq + Hkv) * D:width].reshape(T, Hkv, D)
    if rot:
        wantq = ref.rotate(wantq, pos, rot, interleaved, freq)
        wantk = ref.rotate(wantk, pos, rot, interleaved, freq)
    # fp32 rotation of two operands up to 2^3, sines to 2^-22
    slack = 2.0 ** -18
    err = (q_out.cpu().double().view(T, Hq, D) - wantq).abs()[kept]
    assert bool((err <= wantq.abs()[kept] * ref.HALF_STEP["bf16"] + slack).all())
    old = {"K": c["K"].float().double(), "V": c["V"].float().double()}
    for name, got, want, scale in (("K", K, wantk, c["ks"]), ("V", V, wantv, c["vs"])):
        scale = scale.double()[:, None]
        touched = torch.zeros(got.shape[0], page, dtype=torch.bool)
        for t in range(T):
            if pos[t] < 0:
                continue
            pg, sl = int(c["table"][seq[t], pos[t] // page]), int(pos[t]) % page
            touched[pg, sl] = True
            w = want[t] / scale
            if kv == "e4m3":
                w = w.clamp(-448, 448)
                tol = w.abs() * ref.HALF_STEP["e4m3"] + 2.0 ** -10 + slack / scale
            else:
                tol = w.abs() * ref.HALF_STEP["bf16"] + slack
            assert bool(((got[pg, :, sl] - w).abs() <= tol).all()), (name, t)
        # every other row keeps what it held (NaN where nothing is stored)
        a, b = got.transpose(1, 2)[~touched], old[name].transpose(1, 2)[~touched]
        assert bool(((a == b) | (a.isnan() & b.isnan())).all())


def test_append_far_positions(lib):
    """Angles of far positions: 2^-18 of the exact rotation at position 2^22 + 5."""
    D, page = 64, 16
    far = (1 << 22) + 5
    with tp.Attention(1, 1, D, page) as attn:
        attn.set_rope(D, theta=1e6)
        table = torch.zeros((1, far // page + 1), dtype=torch.int32, device="cuda")
        K = torch.zeros((1, 1, page, D), dtype=torch.bfloat16, device="cuda")
        cache = tp.PagedCache(attn, K, K.clone(), table, torch.tensor([far + 1], dtype=torch.int32, device="cuda"))
        q = queries(1, 1, D, 3)
        got = attn.append(q.cuda(), q.cuda(), q.cuda(), cache, torch.tensor([far], dtype=torch.int32, device="cuda"))
        ok(attn)
    freq = [1e6 ** (-2 * i / D) for i in range(D // 2)]
    want = ref.rotate(q.double().view(1, 1, D), torch.tensor([far]), D, False, freq).view(1, D)
    assert bool(((got.cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -18).all())


def test_append_saturates_and_keeps_nan(lib):
    with tp.Attention(1, 1, 64, 16, kv_dtype="e4m3") as attn:
        K = torch.zeros((1, 1, 16, 64), device="cuda").to(torch.float8_e4m3fn)
        table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        cache = tp.PagedCache(attn, K, K.clone(), table, torch.ones(1, dtype=torch.int32, device="cuda"))
        x = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
        x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1e6, -1e6, math.nan, math.inf
        assert attn.append(None, x, x, cache, torch.zeros(1, dtype=torch.int32, device="cuda")) is None
        ok(attn)
        got = cache.V[0, 0, 0, :5].float().cpu()
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 448 and got[4] == 0


# ------------------------------------------------------------------ decode
SHAPES = [  # Hq, Hkv, D, page, lens, window
    (4, 4, 128, 16, [1, 0, 17, 300, 16], 0),
    (12, 12, 64, 16, [777], 0),
    (32, 8, 128, 64, [1, 129, 128, 127, 2, 0, 515], 0),
    (8, 1, 64, 32, [1000, 31, 33], 0),
    (24, 2, 128, 32, [5, 64, 1023], 0),      # 12 query heads to a kv head
    (40, 1, 128, 128, [260, 1], 0),          # 40: three blocks of query heads
    (18, 2, 64, 256, [511, 3], 0),           # 9
    (6, 2, 128, 16, [1, 40, 333, 0], 33),    # windows
    (16, 4, 64, 64, [200, 64, 65], 64),
    (4, 2, 128, 32, [100, 7], 1),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,window", SHAPES)
def test_decode_matches_definition(lib, kv, Hq, Hkv, D, page, lens, window):
    c = ref.make(Hkv, D, page, kv, lens, seed=Hq + D)
    B = len(lens)
    q = queries(B, Hq, D, page)
    scale = 1.0 / math.sqrt(D)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        wide = torch.zeros((B, Hq * D + 16), dtype=torch.bfloat16, device="cuda")
        wide[:, :Hq * D] = q.cuda()
        out = torch.full((B, Hq * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        got, lse = attn.decode(wide[:, :Hq * D], cache, window=window, out=out[:, :Hq * D], return_lse=True)
        ok(attn)
        assert bool((out[:, Hq * D:] == 7.0).all())
        again, lse2 = attn.decode(q.cuda(), cache, window=window, return_lse=True)
        ok(attn)
        assert torch.equal(again, got) and torch.equal(lse, lse2)  # deterministic
    spans = [(b, b, max(0, n - window) if window else 0, n) for b, n in enumerate(lens)]
    check_rows(c, q, got, lse, spans, Hq, D, scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_long_sequence_is_split_and_joined(lib, kv):
    c = ref.make(2, 128, 64, kv, [20001, 3], seed=9)
    q = queries(2, 8, 128, 9) * 3  # peaked weights
    with tp.Attention(8, 2, 128, 64, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        got, lse = attn.decode(q.cuda(), cache, return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, [(0, 0, 0, 20001), (1, 1, 0, 3)], 8, 128, 128 ** -0.5)


def test_decode_many_sequences(lib):
    """More sequences than a block has threads, lengths 0 to 40."""
    lens = [(7 * b) % 41 for b in range(700)]
    c = ref.make(1, 64, 16, "bf16", lens, seed=4)
    q = queries(700, 3, 64, 4)
    with tp.Attention(3, 1, 64, 16) as attn:
        got, lse = attn.decode(q.cuda(), on_device(c, attn), return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, [(b, b, 0, n) for b, n in enumerate(lens)], 3, 64, 0.125)


def test_decode_reads_lengths_on_replay_and_other_streams(lib):
    """A captured call replays with new lengths and queries; a side stream gives the same."""
    lens = [400, 90, 1]
    c = ref.make(2, 128, 32, "bf16", lens, seed=5)
    q = queries(3, 4, 128, 5)
    with tp.Attention(4, 2, 128, 32) as attn:
        cache = on_device(c, attn)
        qd, out = q.cuda(), torch.empty((3, 512), dtype=torch.bfloat16, device="cuda")
        lse = None
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.decode(qd, cache, out=out)
        for now in (lens, [33, 0, 1], [256, 90, 0]):
            cache.lens.copy_(torch.tensor(now, dtype=torch.int32))
            graph.replay()
            ok(attn)
            want, lse = attn.decode(qd, cache, return_lse=True)
            ok(attn)
            assert torch.equal(out, want)
            check_rows(c, q, out, lse, [(b, b, 0, n) for b, n in enumerate(now)], 4, 128, 128 ** -0.5)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = attn.decode(qd, cache, stream=side)
        side.synchronize()
        assert torch.equal(got, out)


WIDE = [  # more than 8 query heads to a kv head
    (24, 2, 128, 16, [1, 40, 333, 0], 33),
    (40, 2, 64, 64, [129, 0, 1, 700, 65], 0),
    (17, 1, 128, 32, [20, 2000], 129),
    (128, 1, 64, 128, [300, 5], 0),          # the widest group
    (10, 1, 64, 16, [100, 17], 16),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,window", WIDE)
def test_decode_wide_groups(lib, kv, Hq, Hkv, D, page, lens, window):
    test_decode_matches_definition(lib, kv, Hq, Hkv, D, page, lens, window)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_wide_groups_many_and_long(lib, kv):
    lens = [(7 * b) % 41 for b in range(600)]
    lens[77] = 9000
    c = ref.make(1, 64, 16, kv, lens, seed=14)
    q = queries(600, 20, 64, 14)
    with tp.Attention(20, 1, 64, 16, kv_dtype=kv) as attn:
        got, lse = attn.decode(q.cuda(), on_device(c, attn), return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, [(b, b, 0, n) for b, n in enumerate(lens)], 20, 64, 0.125)


# ------------------------------------------------------------------ prompt
def prompt_spans(lens, new, window):
    spans, r = [], 0
    for b, (m, n) in enumerate(zip(lens, new)):
        for i in range(n):
            hi = max(0, m - n + i + 1)
            spans.append((r, b, max(0, hi - window) if window else 0, hi))
            r += 1
    return spans


PROMPTS = [  # Hq, Hkv, D, page, lens, new, window
    (4, 4, 128, 16, [61], [61], 0),
    (12, 12, 64, 16, [1, 130, 0, 300], [1, 130, 0, 17], 0),
    (8, 2, 128, 64, [257, 64, 5], [129, 64, 2], 0),
    (24, 2, 128, 32, [200, 33], [90, 33], 0),      # 12 query heads to a kv head
    (40, 1, 64, 128, [150], [70], 0),
    (6, 2, 64, 16, [3, 50], [5, 50], 0),           # two queries before the first key
    (4, 1, 128, 32, [300, 100], [200, 100], 50),
    (2, 2, 64, 256, [600], [600], 129),
    (3, 1, 128, 64, [515, 1], [515, 1], 0),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new,window", PROMPTS)
def test_prompt_matches_definition(lib, kv, Hq, Hkv, D, page, lens, new, window):
    c = ref.make(Hkv, D, page, kv, lens, seed=Hq + D + 1)
    T = sum(new) + 3  # three rows that belong to no sequence
    q = queries(T, Hq, D, page)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        wide = torch.zeros((T, Hq * D + 24), dtype=torch.bfloat16, device="cuda")
        wide[:, :Hq * D] = q.cuda()
        out = torch.full((T, Hq * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        got, lse = attn.prompt(wide[:, :Hq * D], cu, cache, window=window, out=out[:, :Hq * D], return_lse=True)
        ok(attn)
        assert bool((out[:, Hq * D:] == 7.0).all()) and bool((out[-3:] == 7.0).all())
        again = attn.prompt(q.cuda(), cu, cache, window=window)
        ok(attn)
        assert torch.equal(again[:-3], got[:-3])
    check_rows(c, q, got, lse, prompt_spans(lens, new, window), Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new,window", [
    (8, 2, 128, 64, [9001], [3], 0),               # few queries, many keys: split and joined
    (4, 1, 64, 16, [20011, 5, 0, 129], [40, 2, 0, 129], 0),
    (4, 4, 128, 128, [7000, 7000], [300, 17], 3000),
])
def test_prompt_splits_long_sequences(lib, kv, Hq, Hkv, D, page, lens, new, window):
    c = ref.make(Hkv, D, page, kv, lens, seed=17)
    q = queries(sum(new), Hq, D, 17) * 2
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        got, lse = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
        ok(attn)
        for _ in range(3):  # deterministic, and the counters are back at 0
            assert torch.equal(attn.prompt(q.cuda(), cu, cache, window=window), got)
        ok(attn)
    spans = prompt_spans(lens, new, window)
    check_rows(c, q, got, lse, spans[:6] + spans[6::23] + spans[-3:], Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prompt_many_items(lib, kv):
    """More items than a block tabulates (whole items, dealt in rounds): rows checked in part."""
    lens, new = [3300, 50, 700], [3000, 50, 699]
    Hq, Hkv, D = 96, 12, 64
    c = ref.make(Hkv, D, 32, kv, lens, seed=18)
    q = queries(sum(new), Hq, D, 18)
    cu = torch.tensor([0, 3000, 3050, 3749], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, 32, kv_dtype=kv) as attn:
        got, lse = attn.prompt(q.cuda(), cu, on_device(c, attn), return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, prompt_spans(lens, new, 0)[::97], Hq, D, 0.125)


def test_prompt_many_sequences(lib):
    """More sequences than the table of sequences has entries."""
    lens = [(5 * b) % 23 for b in range(1500)]
    new = [min(n, (3 * b) % 7) for b, n in enumerate(lens)]
    c = ref.make(1, 64, 16, "bf16", lens, seed=19)
    q = queries(sum(new), 2, 64, 19)
    cu = torch.tensor([sum(new[:b]) for b in range(1501)], dtype=torch.int32).cuda()
    with tp.Attention(2, 1, 64, 16) as attn:
        got, lse = attn.prompt(q.cuda(), cu, on_device(c, attn), return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, prompt_spans(lens, new, 0), 2, 64, 0.125)


def test_prompt_replays_with_other_lengths(lib):
    lens, new = [300, 90], [100, 90]
    c = ref.make(2, 128, 32, "bf16", lens, seed=20)
    q = queries(190, 4, 128, 20)
    with tp.Attention(4, 2, 128, 32) as attn:
        cache = on_device(c, attn)
        qd, out = q.cuda(), torch.empty((190, 512), dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor([0, 100, 190], dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.prompt(qd, cu, cache, out=out)
        for now, n in ((lens, new), ([200, 20], [170, 20]), ([0, 90], [0, 1])):
            cache.lens.copy_(torch.tensor(now, dtype=torch.int32))
            cu.copy_(torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32))
            out.fill_(7.0)
            graph.replay()
            ok(attn)
            want, lse = attn.prompt(qd, cu, cache, return_lse=True)
            ok(attn)
            assert torch.equal(out[:sum(n)], want[:sum(n)]) and bool((out[sum(n):] == 7.0).all())
            check_rows(c, q, out, lse, prompt_spans(now, n, 0)[::7], 4, 128, 128 ** -0.5)


# ------------------------------------------------------------------ bad tables
def test_bad_pages_are_left_out_and_reported(lib):
    """A page outside the pool: its keys are left out of decode and prompt, append drops the
    token; every call says so in the status and the context stays usable. The page numbers are
    checked against the pool before any address is made from them."""
    lens = [70, 40]
    c = ref.make(2, 64, 16, "bf16", lens, seed=6)
    q = queries(2, 4, 64, 6)
    with tp.Attention(4, 2, 64, 16) as attn:
        cache = on_device(c, attn)
        good = attn.decode(q.cuda(), cache)
        ok(attn)
        for bad in (-5, c["K"].shape[0], 1 << 30):
            cache.page_table[0, 4] = bad  # keys 64..69
            got, lse = attn.decode(q.cuda(), cache, return_lse=True)
            torch.cuda.synchronize()
            assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
            check_rows(c, q, got, lse, [(0, 0, 0, 64), (1, 1, 0, 40)], 4, 64, 0.125)
            cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
            got, lse = attn.prompt(q.cuda(), cu, cache, return_lse=True)
            torch.cuda.synchronize()
            assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
            check_rows(c, q, got, lse, [(0, 0, 0, 64), (1, 1, 0, 40)], 4, 64, 0.125)
            k = q[:, :128].cuda()
            before = cache.K.clone()
            attn.append(None, k, k, cache, torch.tensor([66, -1], dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
            assert torch.equal(before.view(torch.int16), cache.K.view(torch.int16))
        cache.page_table[0, 4] = int(c["table"][0, 4])
        # positions and sequences outside the table
        for pos, seq in (([80, -1], [0, 0]), ([0, -1], [2, 0]), ([0, -1], [-1, 0])):
            attn.append(None, k, k, cache, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                        torch.tensor(seq, dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
        # a length above the table's capacity counts as the capacity (80 keys)
        cache.lens[0] = 81
        attn.decode(q.cuda(), cache)
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
        cache.lens[0] = 70
        assert torch.equal(attn.decode(q.cuda(), cache), good)
        ok(attn)


# ------------------------------------------------------------------ what a window leaves behind
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new,window", [
    (4, 2, 128, 16, [900, 300], [200, 40], 100),
    (4, 4, 64, 64, [513, 130], [1, 64], 33),
    (2, 1, 128, 256, [700], [300], 50),
    (12, 1, 64, 32, [400, 65, 9000], [17, 65, 3], 1),
    (3, 3, 128, 128, [1000], [500], 131),
])
def test_keys_before_every_window_are_not_used(lib, kv, Hq, Hkv, D, page, lens, new, window):
    """Keys and values that lie before every query's window are NaN, and table entries of pages that
    hold nothing else name no page: results are as ever, and no status is raised."""
    c = ref.make(Hkv, D, page, kv, lens, seed=31)
    K, V, table = c["K"].float(), c["V"].float(), c["table"].clone()

    def poison(firsts):
        for b, first in enumerate(firsts):
            for key in range(first):
                at = int(c["table"][b, key // page])
                K[at, :, key % page] = math.nan
                V[at, :, key % page] = math.nan
            table[b, :first // page] = torch.tensor([-1, 1 << 30])[torch.arange(first // page) % 2].int()
        return dict(c, K=K.to(c["K"].dtype), V=V.to(c["V"].dtype), table=table)

    T, B = sum(new), len(lens)
    q = queries(T, Hq, D, 31)
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(poison([max(0, n - m + 1 - window) for n, m in zip(lens, new)]), attn)
        got, lse = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
        ok(attn)
        spans = prompt_spans(lens, new, window)
        check_rows(c, q, got, lse, spans[:40] + spans[40::7] + spans[-3:], Hq, D, 1.0 / math.sqrt(D))
        cache = on_device(poison([max(0, n - window) for n in lens]), attn)
        got, lse = attn.decode(q[:B].cuda(), cache, window=window, return_lse=True)
        ok(attn)
        check_rows(c, q, got, lse, [(b, b, max(0, n - window), n) for b, n in enumerate(lens)], Hq, D,
                   1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved,T", [
    (1, 1, 64, 16, 64, False, 20001),        # 8 tokens to a block, the last block holds one
    (5, 5, 64, 32, 32, True, 9000),          # 6, dimensions that are not rotated
    (12, 2, 64, 64, 64, False, 5003),        # 4
    (8, 1, 128, 128, 128, False, 5001),      # 4
    (14, 2, 128, 16, 96, True, 2500),        # 2
    (6, 6, 128, 256, 0, False, 2433),
])
def test_append_many_tokens_of_few_heads(lib, kv, Hq, Hkv, D, page, rot, interleaved, T):
    """Blocks of several tokens: as by definition, and the same bits as in small calls."""
    lens = [T // 2 + 9, 1, T - T // 2 + 30]
    c = ref.make(Hkv, D, page, kv, lens, seed=T)
    g = torch.Generator().manual_seed(T)
    q = torch.randn((T, Hq * D), generator=g).bfloat16()
    k = torch.randn((T, Hkv * D), generator=g).bfloat16()
    v = torch.randn((T, Hkv * D), generator=g).bfloat16()
    places = torch.tensor([(b, p) for b, n in enumerate(lens) for p in range(n)], dtype=torch.int32)
    places = places[torch.randperm(len(places), generator=g)[:T]]
    seq, pos = places[:, 0].contiguous(), places[:, 1].contiguous()
    pos[::7] = -1
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        if rot:
            attn.set_rope(rot, interleaved=interleaved)
        whole, parts = on_device(c, attn), on_device(c, attn)
        d = [x.cuda() for x in (q, k, v, pos, seq)]
        out = torch.full((T, Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
        attn.append(*d[:3], whole, d[3], d[4], q_out=out)
        ok(attn)
        small = torch.full_like(out, 7.0)
        for i in range(0, T, 1000):
            x = [y[i:i + 1000] for y in d]
            attn.append(*x[:3], parts, x[3], x[4], q_out=small[i:i + 1000])
        ok(attn)
        assert torch.equal(out, small)
        assert torch.equal(whole.K.view(torch.uint8), parts.K.view(torch.uint8))
        assert torch.equal(whole.V.view(torch.uint8), parts.V.view(torch.uint8))
        kept = pos >= 0
        assert bool((out.cpu()[~kept] == 7.0).all())
        K, V = whole.K.cpu().float().double(), whole.V.cpu().float().double()
    freq = [1e4 ** (-2 * i / rot) for i in range(rot // 2)] if rot else []
    wantq, wantk = q.double().view(T, Hq, D), k.double().view(T, Hkv, D)
    if rot:
        wantq = ref.rotate(wantq, pos, rot, interleaved, freq)
        wantk = ref.rotate(wantk, pos, rot, interleaved, freq)
    slack = 2.0 ** -18
    err = (out.cpu().double().view(T, Hq, D) - wantq).abs()[kept]
    assert bool((err <= wantq.abs()[kept] * ref.HALF_STEP["bf16"] + slack).all())
    pages = c["table"][seq[kept].long(), (pos[kept] // page).long()].long()
    for got, want, scale in ((K, wantk, c["ks"]), (V, v.double().view(T, Hkv, D), c["vs"])):
        scale = scale.double()[:, None]
        w = want[kept] / scale
        if kv == "e4m3":
            w = w.clamp(-448, 448)
            tol = w.abs() * ref.HALF_STEP["e4m3"] + 2.0 ** -10 + slack / scale
        else:
            tol = w.abs() * ref.HALF_STEP["bf16"] + slack
        assert bool(((got[pages, :, (pos[kept] % page).long()] - w).abs() <= tol).all())


def test_append_many_tokens_reports_bad_places(lib):
    """Blocks of several tokens: a bad place drops its own token's k and v only."""
    T, D, page = 4000, 64, 16
    c = ref.make(1, D, page, "bf16", [T], seed=51)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(51)).bfloat16()
    pos = torch.arange(T, dtype=torch.int32)
    with tp.Attention(1, 1, D, page) as attn:
        cache = on_device(c, attn)
        seq = torch.zeros(T, dtype=torch.int32)
        bad = torch.tensor([5, 6, 1000, 3999])
        pos[5], pos[1000] = 1 << 20, T + page
        seq[6], seq[3999] = 1, -1
        before = cache.V.clone()
        got = attn.append(x.cuda(), x.cuda(), x.cuda(), cache, pos.cuda(), seq.cuda())
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
        assert torch.equal(got.cpu(), x)  # queries are written all the same
        good = torch.ones(T, dtype=torch.bool)
        good[bad] = False
        at = torch.arange(T)
        pages = c["table"][0, at // page].long()
        now, old = cache.V.cpu()[pages, 0, at % page], before.cpu()[pages, 0, at % page]
        assert torch.equal(now[good], x[good]) and torch.equal(now[~good], old[~good])
