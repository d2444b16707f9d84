"""The sequence pool's definition in plain Python lists, one block at a time, for
tests of batches that are planned on the GPU."""

import numpy as np
import torch

from paged_kv_cache_56_gb300 import pkv


class PoolModel:
    def __init__(self, max_slots, max_blocks, num_blocks, bs, int8=False, order=None):
        self.max_slots, self.max_blocks, self.N, self.bs, self.int8 = max_slots, max_blocks, num_blocks, bs, int8
        self.lists = [[] for _ in range(max_slots)]
        self.lens = [0] * max_slots
        self.free = list(range(num_blocks)) if order is None else list(order)

    def plan(self, slots, counts, num_tokens, max_tokens):
        """The plan's arrays as a dict, or the error bits."""
        bad, seen, need = 0, set(), 0
        for s, n in zip(slots, counts):
            if s == -1:
                continue
            if not 0 <= s < self.max_slots:
                bad |= pkv.PKV_DEVERR_SLOT
                continue
            if s in seen:
                bad |= pkv.PKV_DEVERR_SLOT
            seen.add(s)
            if not 0 <= n <= max_tokens:
                bad |= pkv.PKV_DEVERR_BATCH
                continue
            blocks = -(-(self.lens[s] + n) // self.bs)
            if blocks > self.max_blocks:
                bad |= pkv.PKV_DEVERR_CTX_LEN
                continue
            need += max(0, blocks - len(self.lists[s]))
        if bad == 0:  # (otherwise which sums the kernel took does not matter)
            if sum(n for s, n in zip(slots, counts) if s != -1) > num_tokens:
                bad |= pkv.PKV_DEVERR_BATCH
            if need > len(self.free):
                bad |= pkv.PKV_DEVERR_OOM
        if bad:
            return bad
        B = len(slots)
        p = dict(starts=[0], tables=np.full((B, self.max_blocks), -1), ctx=[], fill=[], ids=[], off=[], slot=[], pos=[])
        for b, (s, n) in enumerate(zip(slots, counts)):
            if s == -1:
                p["starts"].append(p["starts"][-1])
                p["ctx"].append(0)
                p["fill"].append(-1)
                continue
            while len(self.lists[s]) * self.bs < self.lens[s] + n:
                self.lists[s].append(self.free.pop(0))
            p["tables"][b, :len(self.lists[s])] = self.lists[s]
            end = self.lens[s] + n
            for t in range(self.lens[s], end):
                p["ids"].append(self.lists[s][t // self.bs])
                p["off"].append(t % self.bs)
                p["slot"].append(s)
                p["pos"].append(t)
            p["starts"].append(p["starts"][-1] + n)
            p["ctx"].append(end)
            p["fill"].append(self.lists[s][end // self.bs - 1] if n and end % self.bs == 0 else -1)
        rest = num_tokens - len(p["ids"])
        for name, fill in (("ids", -1), ("off", 0), ("slot", -1), ("pos", 0)):
            p[name] += [fill] * rest
        return p

    def commit(self, slots, counts, accepted):
        bad = 0
        for s, n, a in zip(slots, counts, accepted):
            if s == -1 or n == 0:
                continue
            end, ctx = self.lens[s] + a, self.lens[s] + n
            if not 0 <= a <= n or (self.int8 and end % self.bs and end // self.bs != ctx // self.bs):
                bad |= pkv.PKV_DEVERR_CTX_LEN
                continue
            self.lens[s] = end
        return bad

    def release(self, slots):
        if any(s != -1 and not 0 <= s < self.max_slots for s in slots) or \
                len({s for s in slots if s != -1}) != sum(s != -1 for s in slots):
            return pkv.PKV_DEVERR_SLOT
        for s in slots:
            if s != -1:
                self.free += self.lists[s]
                self.lists[s], self.lens[s] = [], 0
        return 0


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


class DevicePoolOf:
    """A pool on the GPU in the state of a PoolModel, and a plan's arrays. `head`:
    where the ring begins; `wide` False: tables that start off a 16-byte boundary."""

    def __init__(self, m: PoolModel, B, num_tokens, max_tokens, head=0, wide=True):
        self.m, self.B, self.num_tokens = m, B, num_tokens
        tables = np.full((m.max_slots, m.max_blocks), -1, np.int32)
        for s, x in enumerate(m.lists):
            tables[s, :len(x)] = x
        ring = np.full(m.N, -7, np.int32)
        ring[(head + np.arange(len(m.free))) % m.N] = m.free

        def array(x):
            x = np.asarray(x, np.int32)
            t = torch.empty(x.size + 1, dtype=torch.int32, device="cuda")[0 if wide else 1:][:x.size].view(x.shape)
            return t.copy_(torch.as_tensor(x))
        self.tables, self.lens, self.held = array(tables), dev(m.lens), dev([len(x) for x in m.lists])
        self.ring, self.state, self.err = dev(ring), dev([head, len(m.free), 0, 0]), dev([0])
        self.pool = pkv.make_seq_pool(self.tables, self.lens, self.held, self.ring, self.state, block_size=m.bs,
                                      int8=m.int8, err=self.err)
        self.out = dict(starts=array(np.full(B + 1, -9)), tables=array(np.full((B, m.max_blocks), -9)),
                        ctx=array(np.full(B, -9)), fill=array(np.full(B, -9)),
                        **{n: array(np.full(num_tokens, -9)) for n in ("ids", "off", "slot", "pos")})
        o = self.out
        self.plan_desc = pkv.make_plan(o["starts"], o["tables"], o["ctx"], num_tokens=num_tokens, max_tokens=max_tokens,
                                       fill_blocks=o["fill"], block_ids=o["ids"], offsets=o["off"], token_slots=o["slot"],
                                       positions=o["pos"])

    def error(self):
        bits = int(self.err.item())
        self.err.zero_()
        return bits

    def check_state(self):
        m = self.m
        head, free = self.state[:2].tolist()
        assert self.state[2:].tolist() == [0, 0]
        assert self.lens.tolist() == m.lens and self.held.tolist() == [len(x) for x in m.lists]
        assert free == len(m.free)
        ring = self.ring.cpu().numpy()
        assert ring[(head + np.arange(free)) % m.N].tolist() == m.free
        tables = self.tables.cpu().numpy()
        for s, x in enumerate(m.lists):
            assert tables[s, :len(x)].tolist() == x

    def check_plan(self, want):
        for name, x in want.items():
            got = self.out[name].cpu().numpy()
            assert np.array_equal(got, np.asarray(x, np.int32).reshape(got.shape)), name

    def check_empty_plan(self):
        for name, fill in (("starts", 0), ("tables", -1), ("ctx", 0), ("fill", -1), ("ids", -1), ("off", 0), ("slot", -1),
                           ("pos", 0)):
            assert (self.out[name] == fill).all(), name
