"""GPU tests of the router in front of the pool: logits -> route -> ids and weights ->
prepare + forward, on both slot managers, eagerly and replayed from a graph."""
import numpy as np
import pytest
import torch

from _gpu_helpers import DEV, Rig, check_close, from_dev_act, to_dev_act
from expert_slot_cache_amd import binding, synth
from oracle import rows as orows
from oracle.lru import LayerLRU

pytestmark = pytest.mark.gpu

TINY = synth.WORKLOADS["tiny_f32_e8"]
WORKLOADS = {
    "f32": TINY.with_(experts=24, top_k=4, hidden=128, inter=64, slots=10),
    "bf16": TINY.with_(experts=40, top_k=6, hidden=256, inter=128, slots=16, wtype="bf16", atype="bf16"),
    "int4": TINY.with_(experts=32, top_k=3, hidden=256, inter=128, slots=12, wtype="int4", atype="bf16"),
}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def logits_of(rng, T, E, atype):
    """Router logits of T tokens, as device tensor; an eighth of the experts is masked out."""
    z = rng.normal(size=(T, E)).astype(np.float32) + 1.5 * np.sin(np.arange(E, dtype=np.float32))
    z[:, ::8] = -np.inf
    return torch.from_numpy(z).to(TYPES[atype]).to(DEV)


class Buffers:
    def __init__(self, wl, T):
        self.logits = torch.zeros((T, wl.experts), dtype=TYPES[wl.atype], device=DEV)
        self.ids = torch.zeros((T, wl.top_k), dtype=torch.int32, device=DEV)
        self.w = torch.zeros((T, wl.top_k), device=DEV)
        self.slots = torch.zeros_like(self.ids)
        self.x = torch.zeros((T, wl.hidden), dtype=TYPES[wl.atype], device=DEV)
        self.out = torch.zeros_like(self.x)


def check(wl, rig, lru, b, x, what):
    """b's ids, weights and outputs against the oracles; the step's path and misses too."""
    z = b.logits.double().cpu().numpy()
    ids, w = orows.route(z, wl.top_k, True)
    assert np.array_equal(b.ids.cpu().numpy(), ids), what
    assert not (ids % 8 == 0).any(), what             # no masked expert
    r = lru.step(ids)
    assert rig.pool.last_step(0) == (r.path, r.misses), what
    assert np.array_equal(b.slots.cpu().numpy(), r.slot_ids), what
    check_close(from_dev_act(b.out), rig.reference(0, x, ids, w.astype(np.float32)), wl.atype, wl.wtype, what)


@pytest.mark.parametrize("policy", ["host", "device"])
@pytest.mark.parametrize("kind", list(WORKLOADS))
def test_route_feeds_the_pool(kind, policy):
    wl = WORKLOADS[kind]
    rig = Rig(wl, slots=wl.slots, policy=policy, max_tokens=3)
    lru = LayerLRU(wl.experts, wl.slots)
    rng = np.random.default_rng(5)
    for step in range(24):
        T = 1 + step % 3
        b = Buffers(wl, T)
        x = synth.draw_activations(rng, (T, wl.hidden), wl.atype)
        b.logits.copy_(logits_of(rng, T, wl.experts, wl.atype))
        b.x.copy_(to_dev_act(x, wl.atype))
        binding.route(b.logits, b.ids, b.w)
        rig.pool.prepare(0, b.ids, T, b.slots)
        rig.pool.forward(0, b.x, b.slots, b.w, b.out, T)
        check(wl, rig, lru, b, x, f"step {step}")
    rig.close()


@pytest.mark.parametrize("kind", list(WORKLOADS))
def test_route_and_step_replayed_from_a_graph(kind):
    wl = WORKLOADS[kind]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        rig = Rig(wl, slots=wl.slots, policy="device", one_call=True)
    lru = LayerLRU(wl.experts, wl.slots)
    rng = np.random.default_rng(6)
    b = Buffers(wl, 1)

    def load():
        x = synth.draw_activations(rng, (1, wl.hidden), wl.atype)
        with torch.cuda.stream(side):
            b.logits.copy_(logits_of(rng, 1, wl.experts, wl.atype))
            b.x.copy_(to_dev_act(x, wl.atype))
        side.synchronize()
        return x

    def record():
        binding.route(b.logits, b.ids, b.w)
        rig.pool.step(0, b.ids, 1, b.slots, b.x, b.w, b.out)

    torch.cuda.synchronize()
    x = load()
    with torch.cuda.stream(side):
        record()
    side.synchronize()
    check(wl, rig, lru, b, x, "eager")
    g = torch.cuda.CUDAGraph()
    x = load()
    with torch.cuda.graph(g, stream=side):
        record()
    for step in range(12):
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        check(wl, rig, lru, b, x, f"replay {step}")
        torch.cuda.synchronize()
        x = load()
    g.reset()
    rig.close()
