"""GPU: the bits of a pair's row in a routed product through group-scaled weights depend on the weights, the
pair's image row and the sizes of the projections alone: not on the live count, on the bucket or on the routes
of other rows (a captured graph replays a token's step with the same bits, whatever shares the bucket)."""
import numpy as np
import pytest

from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from oracle import oracle as O
from tests.gpu_helpers import dev, host, live_ptr

pytestmark = pytest.mark.gpu

SENTINEL = -12345.5


def expert_weights(seed, G, E, N, K):
    """Packed random experts, made on the device (their values do not matter, their bits do)."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    per = qk.qk_weight_packed_bytes(f"q4_g{G}", N, K)
    out = torch.empty((E * per,), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randint(0, 256, (N, K // G, 4 + G // 2), dtype=torch.uint8, device="cuda", generator=gen)
        w[..., 0:2] = (torch.rand((N, K // G, 1), device="cuda", generator=gen) * 0.02 + 0.001).half().view(torch.uint8)
        qk.qk_weight_pack(f"q4_g{G}", w, N, K, out[e * per:], per)
    return out


class Routed:
    """E experts of one or two projections (N, K), called for a bucket of rows."""

    def __init__(self, G, E, k, sizes, slots):
        self.G, self.E, self.k, self.sizes, self.slots = G, E, k, sizes, slots
        self.rb = max(K for _, K in sizes) // 32
        self.w = [expert_weights(700 + j, G, E, N, K) for j, (N, K) in enumerate(sizes)]

    def buffers(self, rows):
        import torch
        i32 = lambda n: torch.full((n,), -3, dtype=torch.int32, device="cuda")
        b = dict(rows=rows, ids=i32(rows * self.k), counts=i32(self.E), offsets=i32(self.E + 1), items=i32(rows * self.k),
                 img=torch.zeros(((rows * self.k if self.slots else rows) * self.rb * 36,), dtype=torch.uint8, device="cuda"),
                 y=[torch.zeros((rows * self.k, N), device="cuda") for N, _ in self.sizes], live=live_ptr(rows))
        b["projs"] = [qk.make_proj_id(f"q4_g{self.G}", self.E, w, N, K, y)
                      for w, (N, K), y in zip(self.w, self.sizes, b["y"])]
        return b

    def call(self, b):
        qk.qk_moe_plan(b["ids"], b["rows"], self.k, self.E, b["counts"], b["offsets"], b["items"], b["live"])
        (qk.qk_mmvq_id_slots if self.slots else qk.qk_mmvq_id)(b["img"], self.rb, b["rows"], self.k, b["projs"], b["counts"],
                                                               b["offsets"], b["items"])

    def fill(self, b, img, ids, live):
        """The first `live` rows; the rest of the bucket is poison."""
        n = live * self.k if self.slots else live
        b["img"].fill_(0xFF)
        b["img"][:n * self.rb * 36].copy_(dev(img[:n].reshape(-1)))
        b["ids"].fill_(0)
        b["ids"][:live * self.k].copy_(dev(ids[:live].reshape(-1)))
        b["live"].fill_(live)
        for y in b["y"]:
            y.fill_(SENTINEL)

    def run(self, b, img, ids, live):
        self.fill(b, img, ids, live)
        self.call(b)
        assert qk.qk_device_faults() == 0
        return [host(y).copy() for y in b["y"]]


CASES = [
    # group, experts, k, (N, K) of the projections, slots, bucket, live counts
    (64, 128, 8, ((768, 2560), (768, 2560)), False, 16, (1, 2, 5, 9, 13)),
    (128, 128, 8, ((512, 768),), True, 32, (1, 3, 10, 21)),
    (64, 8, 2, ((257, 4096), (40, 1024)), False, 24, (1, 2, 4, 8, 17)),
    (128, 4, 1, ((96, 9344),), False, 16, (1, 2, 7)),            # more columns than one CTA's fragments hold
    (64, 16, 4, ((33, 192),), True, 64, (1, 6, 40)),
    (128, 3, 2, ((1500, 1024),), False, 200, (1, 16, 120)),      # several passes per expert
]


@pytest.mark.parametrize("G,E,k,sizes,slots,bucket,lives", CASES)
def test_bits_do_not_depend_on_live_count_bucket_or_other_routes(G, E, k, sizes, slots, bucket, lives):
    import torch
    m = Routed(G, E, k, sizes, slots)
    g = synth.rng(31 + E + bucket)
    ids = np.stack([g.permutation(E)[:k] for _ in range(bucket)]).astype(np.int32)
    img = O.quantize_q8_1(synth.activations(32 + bucket, bucket * k if slots else bucket, m.rb * 32)).reshape(
        bucket * k if slots else bucket, -1)
    b = m.buffers(bucket)
    full = m.run(b, img, ids, bucket)
    bits = lambda a: a.view(np.uint32)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        m.call(b)
    for live in lives:
        m.fill(b, img, ids, live)
        torch.cuda.synchronize()
        graph.replay()
        got = [host(y).copy() for y in b["y"]]
        exact = m.run(m.buffers(live), img, ids, live)          # a bucket of just these rows
        for full_j, got_j, exact_j in zip(full, got, exact):
            assert np.array_equal(bits(got_j[:live * k]), bits(full_j[:live * k])), f"replay at live {live}"
            assert np.array_equal(bits(exact_j), bits(full_j[:live * k])), f"bucket of {live} rows"
            assert np.all(got_j[live * k:] == SENTINEL)
    # the first row keeps its routes, all others go to one expert
    other = ids.copy()
    other[1:] = ids[0, 0]
    for full_j, got_j in zip(full, m.run(b, img, other, bucket)):
        assert np.array_equal(bits(got_j[:k]), bits(full_j[:k]))
