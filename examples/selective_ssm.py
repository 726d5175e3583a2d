"""A small stack of selective state space layers served from state slots.

Three requests go through the calls of a serving engine: prompts of different
lengths in one packed prefill, with checkpoints; a request that shares a prefix
and starts from a fork of its checkpoint; speculative steps, in which drafts are
rejected now and then; the end of a request, its slot freed and the others moved
down.  The outputs are compared with one prefill of each whole text.

    python examples/selective_ssm.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from recurrent_kda_state_gb300 import kda as K  # noqa: E402

LAYERS, MODEL, INNER, STATE, WIDTH, RANK, VOCAB = 3, 256, 512, 16, 4, 16, 997
SLOTS, EVERY = 12, 64  # state slots, tokens between checkpoints
BF16 = torch.bfloat16


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Layer:
    """One layer's weights and its two pools."""

    def __init__(self, gen):
        def w(*shape, std=None):
            std = shape[-1] ** -0.5 if std is None else std
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF16)
        self.inp, self.out = w(2 * INNER, MODEL), w(MODEL, INNER)
        self.proj, self.dt = w(RANK + 2 * STATE, INNER), w(INNER, RANK)
        self.taps, self.bias = w(INNER, WIDTH, std=WIDTH ** -0.5), w(INNER, std=0.1)
        step = torch.exp(torch.rand(INNER, generator=gen, device="cuda") * 4.6 - 6.9)
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.A = -torch.arange(1, STATE + 1, device="cuda").float().repeat(INNER, 1)
        self.D = torch.ones(INNER, device="cuda")
        self.conv = K.ConvPool.zeros(SLOTS, WIDTH, INNER, BF16)
        self.scan = K.ScanPool.zeros(SLOTS, INNER, STATE)

    def __call__(self, x, cu, slots, commit=None, ckpt=None, start=None, step=False):
        """x [N][MODEL] packed rows -> the layer's output, the slots moved on."""
        xz = x @ self.inp.T
        conv = K.ConvBatch(xz[:, :INNER], self.taps, self.bias, cu)
        if step:
            K.kda_conv_step(conv, self.conv, slots, commit)
        else:
            K.kda_conv_prefill(conv, self.conv, slots, EVERY if ckpt is not None else 0, ckpt, start)
        u = conv.y
        low = u @ self.proj.T  # time step, B and C of a token
        b, c = (low[:, RANK + k * STATE:RANK + (k + 1) * STATE].unflatten(1, (1, STATE))
                for k in (0, 1))
        scan = K.ScanBatch(u, low[:, :RANK] @ self.dt.T, self.A, b, c, D=self.D,
                           z=xz[:, INNER:], dt_bias=self.dt_bias, cu_seqlens=cu)
        if step:
            K.kda_scan_step(scan, self.scan, slots, commit)
        else:
            K.kda_scan_prefill(scan, self.scan, slots, EVERY if ckpt is not None else 0, ckpt, start,
                               K.scan_workspace(scan))
        return x + scan.y @ self.out.T


class Model:
    def __init__(self, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn(VOCAB, MODEL, generator=gen, device="cuda").to(BF16)
        self.layers = [Layer(gen) for _ in range(LAYERS)]
        self.arrays = K.SlotArrays([t for l in self.layers for t in (l.conv.data, l.scan.data)])

    def __call__(self, rows, slots, **kw):
        """rows: lists of token ids; returns their outputs, a tensor each."""
        lens = [len(r) for r in rows]
        cu = i32([sum(lens[:k]) for k in range(len(lens) + 1)])
        x = self.embed[torch.tensor([t for r in rows for t in r], device="cuda")]
        for layer in self.layers:
            x = layer(x, cu, i32(slots), **kw)
        return list(x.split(lens))

    def move(self, src, dst):
        K.kda_move_slots(self.arrays, i32(src), i32(dst), K.move_workspace(self.arrays, len(dst)))


def main():
    torch.manual_seed(1)
    rng = torch.Generator().manual_seed(2)

    def text(n):
        return torch.randint(VOCAB, (n,), generator=rng).tolist()
    model = Model()
    first, second = text(300), text(171)
    third = first[:128] + text(90)  # shares two blocks of 64 tokens with the first
    texts, prompts = [first, second, third], [200, 101, 160]

    # two prompts in one pass; checkpoints of the first after 64 and 128 tokens
    ckpt = i32([[8, 9], [-1, -1]])
    out = model([first[:200], second[:101]], [0, 1], ckpt=ckpt)
    # the third starts from a fork of the second checkpoint
    model.move([9], [2])
    out += model([third[128:160]], [2], start=i32([128]))
    got = [[out[0]], [out[1]], [out[2]]]

    # speculative steps: a row is what was accepted last time, not yet in the
    # state, and four drafts; every third draft is wrong
    done = list(prompts)          # tokens whose outputs are final
    behind = [0, 0, 0]            # of these, not yet in the state
    slots, live, count = [0, 1, 2], [0, 1, 2], 0
    while live:
        rows, good = [], []
        for r in live:
            drafts = texts[r][done[r]:done[r] + 4]
            ok = 0
            while ok < len(drafts) and (count + ok) % 3 != 2:
                ok += 1
            if ok < len(drafts):  # the wrong draft, then what follows it
                drafts = drafts[:ok] + [(drafts[ok] + 1) % VOCAB] + drafts[ok + 1:]
            count += max(1, ok)
            rows.append(texts[r][done[r] - behind[r]:done[r]] + drafts)
            good.append(ok)
        # a row that is all drafts with none right still needs one true token
        for k, r in enumerate(live):
            if good[k] == 0:
                rows[k] = rows[k][:behind[r]] + texts[r][done[r]:done[r] + 1]
                good[k] = 1
        ys = model(rows, [slots[r] for r in live], commit=i32([behind[r] for r in live]), step=True)
        for k, r in enumerate(live):
            got[r].append(ys[k][behind[r]:behind[r] + good[k]])
            done[r] += good[k]
            behind[r] = good[k]
        ended = [r for r in live if done[r] == len(texts[r])]
        live = [r for r in live if r not in ended]
        if ended:  # free their slots, and move the last live ones down into them
            src, dst = [], []
            keep = sorted(slots[r] for r in live)
            for new, old in enumerate(keep):
                if new != old:
                    src.append(old), dst.append(new)
            freed = [s for s in range(3) if s >= len(keep)]
            model.move(src + [-1] * len(freed), dst + freed)
            for r in live:
                slots[r] = keep.index(slots[r])
    bits = K.kda_get_device_error()

    worst = 0.0
    for r, whole in enumerate(texts):
        model.move([-1], [7])
        mine = torch.cat(got[r]).float()  # the third's from its fork on
        want = model([whole], [7])[0].float()[len(whole) - len(mine):]
        assert len(mine) == len(whole) - (128 if r == 2 else 0)
        worst = max(worst, float((mine - want).norm() / want.norm()))
    print("3 requests, %d tokens: relative difference to whole prefills %.2e, device error %d"
          % (sum(map(len, texts)), worst, bits))
    return worst, bits


if __name__ == "__main__":
    from recurrent_kda_state_gb300._build import build_library
    build_library()
    worst, bits = main()
    sys.exit(0 if worst < 2e-2 and bits == 0 else 1)
