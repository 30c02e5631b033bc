"""The paged 4-bit decode where every CTA has many tiles and several segments to walk, against fp64: reuse of raw, key and
value stages, of score and weight buffers and of the queries' place, partials at both ends of a range, and references that
rise within a segment.  One case at least for each kernel: 16, 32 or 64 rows a unit, d = 128, 256 or 512, tiles copied as
boxes (pages with runs of 16 rows, d <= 256) or loaded by the converters.

That a CTA's walk is long enough follows from counts alone, whatever the partition: with more than k P units (tiles) over P
CTAs, some CTA has more than k."""
import math

import numpy as np
import pytest
import torch

from paged_large_util import decode64, make_large, make_queries, ragged, tiles
from paged_util import D_ROPE, check_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu):
    import latent_kv_cache_split_b200 as lib
    lib.check_device(clear=True)
    return lib


def _sms(gpu):
    return torch.cuda.get_device_properties(gpu).multi_processor_count


def _units(G, H, s_q):
    """Units of a request: groups times blocks of at most 64 rows."""
    return G * -(-(s_q * H // G) // 64)


KERNELS = [
    # d, groups, heads, s_q, page
    (128, 4, 64, 1, 16),     # 16 rows, boxes
    (128, 2, 10, 2, 5),      # 10 of 16 rows, single rows
    (128, 2, 32, 2, 64),     # 32 rows, boxes
    (128, 3, 48, 2, 256),    # 32 rows, boxes of a whole tile, three groups
    (128, 8, 160, 1, 8),     # 20 of 32 rows, single rows
    (128, 1, 40, 1, 32),     # 40 of 64 rows, boxes
    (128, 2, 160, 1, 48),    # 80 rows: two units a group, boxes
    (128, 2, 128, 1, 1),     # 64 rows, single rows
    (256, 4, 32, 2, 16),     # 16 rows, boxes
    (256, 1, 16, 1, 8),      # 16 rows, single rows
    (256, 1, 32, 1, 128),    # 32 rows, boxes
    (256, 2, 48, 1, 100),    # 24 of 32 rows, single rows
    (256, 2, 128, 1, 64),    # 64 rows, boxes
    (256, 1, 100, 2, 24),    # 200 rows: four units a group, single rows
    (512, 2, 16, 2, 16),     # 16 rows
    (512, 1, 30, 1, 64),     # 30 of 32 rows
    (512, 1, 128, 1, 64),    # 128 rows: two units
]


@pytest.mark.parametrize("d,G,H,s_q,page", KERNELS)
def test_many_tiles_and_segments(L, gpu, d, G, H, s_q, page):
    """Results against fp64; the same bits again, and from two streams at once."""
    sms, U = _sms(gpu), _units(G, H, s_q)
    lens = ragged(2 * sms // U + 3, 400, d + G + H, 3000)
    live = sum(n > 0 for n in lens)
    assert U * live > 2 * sms, "some CTA walks three units"
    assert U * tiles(lens) > 6 * sms, "some CTA takes more tiles than twice the stages of any ring"
    pool, table = make_large(lens, G, d, page, H + page, gpu)
    q, qr = make_queries(len(lens), s_q, H, d, H, gpu)
    n, scale = torch.tensor(lens, dtype=torch.int32, device=gpu), 1 / math.sqrt(d + D_ROPE)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full(q.shape[:-1], float("nan"), device=gpu)
    args = (q, qr, pool, G, table, n, scale)
    L.paged_decode_int4(*args, out=out, lse=lse)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    check_decode(out, lse, decode64(q, qr, pool, G, table, lens, scale), d, max(lens), f"d={d} G={G} H={H}")
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(2):
        for s in streams:
            got.append(L.paged_decode_int4(*args, stream=s))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    for o, l in got:
        assert torch.equal(o, out) and torch.equal(l, lse)


# The first column of a tile's RoPE keys; a row with a in that column of its query gets a scale log2(e) of it, in log2 units
# 1.67 (d = 128), 1.29 (256) or 0.96 (512) for 16.
LEVELS = {
    "both": (0, 0, 80, 80, 160, 160, 80, 80),       # up and down by more than 64, for the odd and the even tiles
    "one": (0, 80, 0, 160, 0, 80, 0, 40),           # every second tile alone
    "small": (0, 6, 12, 6, 18, 0, 24, 12),          # by 6 to 40
    "far": (0, 0, 0, 0, 1536, 0, 0, 0),             # by some 1500 to 2500: past what fp32 or bf16 holds as 2^x
}


def _long(gpu, G, H, s_q):
    """Three long requests and an idle one, whose tiles make pieces of more than seven tiles on average."""
    sms, U = _sms(gpu), _units(G, H, s_q)
    per = 7 * (sms + 3 * U) // (3 * U) + 2
    lens = [128 * per, 128 * per - 77, 0, 128 * per - 127]
    # a unit is cut at most once at each range's border, so there are at most P + units pieces
    assert U * tiles(lens) > 7 * (sms + 3 * U)
    return lens


@pytest.mark.parametrize("d,G,H,s_q,page", KERNELS)
@pytest.mark.parametrize("kind", ["both", "one", "small", "far"])
def test_references_rise_within_a_segment(L, gpu, d, G, H, s_q, page, kind):
    """Rows whose scores go up while others' go down, at every change of level, and rows that follow a little of it, whose
    earlier sums still count after a rise."""
    lens, wave = _long(gpu, G, H, s_q), LEVELS[kind]
    at = torch.tensor(wave, device=gpu)
    pool, table = make_large(lens, G, d, page, H + page, gpu, key0=lambda b, t: at[(t // 128 + b) % len(wave)])
    q, qr = make_queries(len(lens), s_q, H, d, H, gpu)
    a = torch.tensor([16.0, 0.0, -16.0, 0.5, -2.0], device=gpu)
    h, i = torch.arange(H, device=gpu), torch.arange(s_q, device=gpu)
    qr[..., 0] = a[(h + 2 * i[:, None]) % 5]
    scale = 1 / math.sqrt(d + D_ROPE)
    out, lse = L.paged_decode_int4(q, qr, pool, G, table, torch.tensor(lens, dtype=torch.int32, device=gpu), scale)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    check_decode(out, lse, decode64(q, qr, pool, G, table, lens, scale), d, max(lens), kind)


@pytest.mark.parametrize("step", [12, 36, 48, 1536])
@pytest.mark.parametrize("exponent", [93, -105])
@pytest.mark.parametrize("d,G,H,s_q,page", [(128, 4, 64, 1, 16), (128, 2, 128, 1, 1), (256, 2, 48, 1, 128), (512, 1, 128, 1, 64)])
def test_values_over_the_cache_s_whole_range(L, gpu, d, G, H, s_q, page, exponent, step):
    """Latents up to 105 2^93, just below 2^100, and scales from 8 2^-105 on, where scores rise by 12 to 1500 and more log2
    units between tiles: sums of weights times values stay finite and keep their precision.  The latent columns of the queries
    are 0, so the scores come from the RoPE keys."""
    lens = _long(gpu, G, H, s_q)
    pool, table = make_large(lens, G, d, page, H + step, gpu, exponent=exponent,
                             key0=lambda b, t: torch.where(t // 128 % 4 == 2, float(step), 0.0))
    q, qr = make_queries(len(lens), s_q, H, d, H, gpu)
    q.zero_()
    qr[..., 0] = 16.0
    scale = 1 / math.sqrt(d + D_ROPE)
    out, lse = L.paged_decode_int4(q, qr, pool, G, table, torch.tensor(lens, dtype=torch.int32, device=gpu), scale)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    ref = decode64(q, qr, pool, G, table, lens, scale)
    back = 2.0 ** (-6 - exponent)      # exact: values as a cache with scales from 8 2^-6 on has them
    check_decode(out.double() * back, lse, (ref[0] * back, ref[1], ref[2] * back, ref[3]), d, max(lens), f"{exponent} {step}")


@pytest.mark.parametrize("d,G,H,s_q,page", [(128, 8, 128, 2, 64), (128, 2, 128, 1, 1), (256, 2, 128, 1, 16), (512, 1, 128, 2, 64)])
def test_every_slot_idle(L, gpu, d, G, H, s_q, page):
    """As in the warm-up of a captured step: zeros and -inf, no table entry read; the captured call then serves requests."""
    B = 200
    lens = [0] * B
    pool, table = make_large([3 * page + 1] * B, G, d, page, 1, gpu)
    q, qr = make_queries(B, s_q, H, d, 2, gpu)
    n = torch.zeros(B, dtype=torch.int32, device=gpu)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full(q.shape[:-1], float("nan"), device=gpu)
    ws = torch.empty(L.paged_decode_workspace_size(B, s_q, H, G, d, _sms(gpu)), dtype=torch.uint8, device=gpu)
    call = lambda: L.paged_decode_int4(q, qr, pool, G, table, n, 0.06, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert L.check_device() == 0
    assert (out == 0).all() and torch.isneginf(lse).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lens[7], lens[150] = 3 * page + 1, 1
    for some in (lens, [0] * B, [-5] * B):
        n.copy_(torch.tensor(some, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert L.check_device() == 0
        check_decode(out, lse, decode64(q, qr, pool, G, table, some, 0.06), d, max(max(some), 1), "replayed")


def test_table_much_wider_than_the_requests(L, gpu):
    """max_pages of a long context, most entries unused."""
    from paged_util import make_pool, queries
    from oracle import paged
    rng = np.random.default_rng(41)
    d, G, H, lens, page = 128, 4, 32, [300, 0, 45], 16
    pool, table = make_pool(rng, lens, G, d, page, max_pages=8192)
    q, qr = queries(rng, 3, 1, H, d)
    out, lse = L.paged_decode_int4(q.to(gpu), qr.to(gpu), torch.from_numpy(pool).to(gpu), G, torch.from_numpy(table).to(gpu),
                                   torch.tensor(lens, dtype=torch.int32, device=gpu), 0.07)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    check_decode(out, lse, paged.paged_decode(q, qr, pool, G, table, lens, 0.07), d, 300)
