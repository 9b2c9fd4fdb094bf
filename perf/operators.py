"""What is measured of the operators around the offset/mask predictor's weight.

The predictor is the one learned layer this package computes: a 1x1 projection
whose output is the aggregation's offset_mask records. Four operators train
and serve it:

  mx          mx_quantize / mx_dequantize: microscaled 4-bit floating point
              (blocks of 32 e2m1 elements that share a power-of-two scale)
  predictor_mx        the projection with both operands in that format, the
              activations quantised on the way, records written as by predictor
  predictor_backward  gradients of the projection's input, weight and bias from
              the fp32 record gradients that backward writes
  orthogonalize       the Newton-Schulz iteration that turns a weight's gradient
              (or momentum) into an orthogonalised update, a stack at a time

``listed()`` names the cases, ``draw`` gives more of the same ranges,
``prepare`` makes a case's inputs, ``run`` makes one pass through an operator
(its plain form, or this package's own where ``own`` is true), ``work`` states
what a pass cannot do without and ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ------------------------------------------------------------------- cases ---

def _mx(name, M, C, dtype):
    return {"name": name, "op": "mx", "M": M, "C": C, "dtype": dtype}


def _pred(name, op, M, C, G, K, dtype, remove_center=False, bias=True):
    return {"name": name, "op": op, "M": M, "C": C, "G": G, "K": K, "dtype": dtype,
            "remove_center": remove_center, "bias": bias}


def _ortho(name, B, R, C, dtype):
    return {"name": name, "op": "orthogonalize", "B": B, "R": R, "C": C, "dtype": dtype}


def listed():
    return [
        # the stage-3 predictor's weight quantised after training (16 groups of 27 channels from 256)
        _mx("mx_stage3_weight_f32", 432, 256, "f32"),
        # the stage-1 activations of a batch of 64 images, quantised and read back (4-bit aware training)
        _mx("mx_stage1_activations_bf16", 64 * 56 * 56, 64, "bf16"),
        # one stage-3 image while serving: latency counts
        _pred("mx_predictor_stage3_one_image_f16", "predictor_mx", 14 * 14, 256, 16, 3, "f16"),
        # the stage-1 batch
        _pred("mx_predictor_stage1_f16", "predictor_mx", 64 * 56 * 56, 64, 4, 3, "f16"),
        # the high-resolution pair of images (254 x 254 outputs)
        _pred("mx_predictor_highres_bf16", "predictor_mx", 2 * 254 * 254, 128, 8, 3, "bf16"),
        # the latent block's width on odd extents, centre point removed, fp32 activations, no bias
        _pred("mx_predictor_latent_odd_f32", "predictor_mx", 7 * 61 * 61, 320, 8, 3, "f32", True, False),
        # training: gradients of one stage-3 image (the smallest batch)
        _pred("predictor_backward_stage3_one_image_f16", "predictor_backward", 14 * 14, 256, 16, 3, "f16"),
        # gradients of the stage-1 batch
        _pred("predictor_backward_stage1_bf16", "predictor_backward", 64 * 56 * 56, 64, 4, 3, "bf16"),
        # the latent block's width on odd extents, centre point removed, in fp32
        _pred("predictor_backward_latent_odd_f32", "predictor_backward", 7 * 61 * 61, 320, 8, 3, "f32", True),
        # the four stage-1 blocks' weights (108 x 64), one update
        _ortho("orthogonalize_stage1_f32", 4, 108, 64, "f32"),
        # the eighteen stage-3 blocks' weights (432 x 256), one update
        _ortho("orthogonalize_stage3_f32", 18, 432, 256, "f32"),
        # the four stage-4 blocks' weights (32 groups: 864 x 512), bf16 momentum
        _ortho("orthogonalize_stage4_bf16", 4, 864, 512, "bf16"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mx", "predictor_mx", "predictor_backward", "orthogonalize"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "mx":
        C = _logint(rng, 1, 512)
        M = _logint(rng, 1, 200704)
        M = max(1, min(M, 200704 * 64 * 2 // (C * SIZES[dtype])))
        return {"op": op, "M": M, "C": C, "dtype": dtype}
    if op == "orthogonalize":
        B, R, C = _logint(rng, 1, 18), _logint(rng, 8, 1024), _logint(rng, 8, 1024)
        B = max(1, min(B, 4 * 864 * 512 * 512 // (R * C * min(R, C))))
        if R * C * min(R, C) > 4 * 864 * 512 * 512:
            C = 512
        return {"op": op, "B": B, "R": R, "C": C, "dtype": dtype}
    K = rng.choice([1, 3, 3, 3, 5])
    remove_center = K == 3 and rng.random() < 0.3
    P = K * K - (1 if remove_center else 0)
    G = _logint(rng, 1, max(1, min(32, 864 // (3 * P))))
    C = _logint(rng, 8, 512)
    NO = 3 * G * P
    # no more than the costliest listed case of the operator, in bytes and in products
    if op == "predictor_mx":
        most, e = 2 * 2 * 254 * 254 * (128 + 216), SIZES[dtype]
        M = min(most // (e * (C + NO)), 2 * 254 * 254 * 128 * 216 // (C * NO))
    else:
        most, e = 64 * 56 * 56 * (64 * 2 + 108 * 4 + 64 * 4), SIZES[dtype]
        M = min(most // (C * e + NO * 4 + C * 4), 7 * 61 * 61 * 320 * 192 // (C * NO))
    M = _logint(rng, 1, max(1, M))
    return {"op": op, "M": M, "C": C, "G": G, "K": K, "dtype": dtype, "remove_center": remove_center,
            "bias": rng.random() < 0.8}


# ------------------------------------------------------------------ inputs ---

def _points(case):
    return case["K"] * case["K"] - (1 if case["remove_center"] else 0)


def _activations(g, M, C, dtype):
    """Activations of a depthwise convolution: channels of different size, a few pixels all zero."""
    dev = torch.device("cuda")
    y = torch.randn(M, C, generator=g, device=dev)
    y *= torch.exp(0.7 * torch.randn(C, generator=g, device=dev))
    y[torch.rand(M, generator=g, device=dev) < 0.01] = 0.0
    return y.to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    state = dict(case)
    if case["op"] == "orthogonalize":
        # a gradient of decaying spectrum over a floor of noise, as momentum buffers have
        B, R, C = case["B"], case["R"], case["C"]
        k = max(1, min(R, C) // 4)
        scale = torch.linspace(0.0, -4.0, k, device=dev).exp()
        x = torch.matmul(torch.randn(B, R, k, generator=g, device=dev) * scale,
                         torch.randn(B, k, C, generator=g, device=dev))
        x += 0.1 * torch.randn(B, R, C, generator=g, device=dev)
        state["x"] = (x * 1e-3).to(DTYPES[case["dtype"]])
        return state
    M, C = case["M"], case["C"]
    if case["op"] == "mx":
        state["x"] = _activations(g, M, C, case["dtype"])
        return state
    NO = 3 * case["G"] * _points(case)
    state["y"] = _activations(g, M, C, case["dtype"])
    w = torch.randn(NO, C, generator=g, device=dev) * C ** -0.5
    if case["op"] == "predictor_mx":
        # the weight is quantised once and kept
        state["codes"], state["scales"] = _encode(w)
        state["bias"] = torch.randn(NO, generator=g, device=dev) if case["bias"] else None
        return state
    state["weight"] = w.to(DTYPES[case["dtype"]])
    # record gradients: pixels of very different size, some without any
    gom = torch.randn(M, case["G"], 3 * _points(case), generator=g, device=dev)
    gom *= 1e-3 * torch.exp(torch.randn(M, 1, 1, generator=g, device=dev))
    gom[torch.rand(M, generator=g, device=dev) < 0.05] = 0.0
    state["grad_offset_mask"] = gom
    return state


# ------------------------------------------------------------- plain forms ---

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(code):
    """2^(code - 127) in fp32 for whole codes 0..254 (code 0: the subnormal 2^-127)."""
    bits = torch.where(code > 0, code << 23, torch.full_like(code, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _blocks(x):
    """x [M, C] as fp32 [M, blocks, 32], zeros past C."""
    M, C = x.shape
    nb = (C + 31) // 32
    xp = torch.zeros(M, nb * 32, dtype=torch.float32, device=x.device)
    xp[:, :C] = x
    return xp.view(M, nb, 32)


def _quantise(x):
    """(element codes [M, blocks, 32] whole numbers 0..15, scale codes [M, blocks])."""
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    exponent = (amax.view(torch.int32) >> 23).long()
    scale = torch.clamp(exponent - 2, min=0)
    q = b * _pow2(254 - scale).unsqueeze(2)
    a = q.abs()
    # round to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    code = ((a > 0.25).long() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code + 8 * torch.signbit(b), scale


def _encode(x):
    """Packed codes uint8 [M, 16*blocks] (element 2i in the low half of byte i), scales uint8 [M, blocks]."""
    code, scale = _quantise(x)
    M = x.shape[0]
    pair = code.view(M, -1, 2)
    return (pair[..., 0] + 16 * pair[..., 1]).to(torch.uint8), scale.to(torch.uint8)


def _value(code, scale):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=code.device)
    return table[code] * _pow2(scale).unsqueeze(2)


def _decode(codes, scales, C):
    M, nb = scales.shape
    c = codes.long()
    code = torch.stack((c & 15, c >> 4), dim=2).view(M, nb, 32)
    return _value(code, scales.long()).view(M, nb * 32)[:, :C]


def _pack(params, G, P):
    """Projection channels [M, 3GP] (all groups' offsets, then all groups' masks) as records [M, G, 3P]."""
    M = params.shape[0]
    return torch.cat((params[:, :2 * G * P].reshape(M, G, 2 * P), params[:, 2 * G * P:].reshape(M, G, P)), dim=2)


def _unpack(records, G, P):
    M = records.shape[0]
    return torch.cat((records[:, :, :2 * P].reshape(M, 2 * G * P), records[:, :, 2 * P:].reshape(M, G * P)), dim=1)


def _plain(state):
    op, dt = state["op"], DTYPES[state["dtype"]]
    if op == "mx":
        x = state["x"]
        code, scale = _quantise(x)
        return _value(code, scale).view(x.shape[0], -1)[:, :x.shape[1]].to(dt), scale.to(torch.uint8)
    if op == "predictor_mx":
        G, P, y = state["G"], _points(state), state["y"]
        w = _decode(state["codes"], state["scales"], state["C"])
        code, scale = _quantise(y)
        q = _value(code, scale).view(y.shape[0], -1)[:, :y.shape[1]]
        params = torch.matmul(q, w.t())
        if state["bias"] is not None:
            params = params + state["bias"]
        return _pack(params, G, P).to(dt)
    if op == "predictor_backward":
        gp = _unpack(state["grad_offset_mask"], state["G"], _points(state))
        grad_y = torch.matmul(gp, state["weight"].float())
        grad_w = torch.matmul(gp.t(), state["y"].float())
        # the bias sums every pixel: 64 bits keep the long sum
        grad_b = gp.sum(dim=0, dtype=torch.float64).float() if state["bias"] else None
        return [grad_y, grad_w] + ([grad_b] if state["bias"] else [])
    x = state["x"].float()
    a, b, c = COEFFICIENTS
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = x / (norm + EPS).float()
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if tall:
        x = x.transpose(1, 2)
    return x.to(dt).contiguous()


def _own(state):
    import deformable_convolution_sparse_b200 as dcn
    op = state["op"]
    if op == "mx":
        x = state["x"]
        codes, scales = dcn.mx_quantize(x)
        return dcn.mx_dequantize(codes, scales, x.shape[1], x.dtype), scales
    if op == "predictor_mx":
        return dcn.predictor_mx(state["y"], state["codes"], state["scales"], state["bias"], G=state["G"],
                                K=state["K"], remove_center=state["remove_center"])
    if op == "predictor_backward":
        grads = dcn.predictor_backward(state["y"], state["weight"], state["grad_offset_mask"], G=state["G"],
                                       K=state["K"], remove_center=state["remove_center"],
                                       with_bias=state["bias"])
        return list(grads[:3 if state["bias"] else 2])
    return dcn.orthogonalize(state["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ---

def work(case):
    """Inputs read once, outputs written once, the products of the formulas."""
    e = SIZES[case["dtype"]]
    if case["op"] == "orthogonalize":
        B, R, C = case["B"], case["R"], case["C"]
        n, m = min(R, C), max(R, C)
        return {"bytes": 2 * B * R * C * e, "flops": B * STEPS * (2 * n * n * m + 2 * n * n * n + 2 * n * n * m)}
    M, C = case["M"], case["C"]
    nb = (C + 31) // 32
    if case["op"] == "mx":
        # quantise: x in, codes and scales out; read back: those in, values out
        return {"bytes": 2 * (M * C * e + M * nb * 17), "flops": 4 * M * C}
    NO = 3 * case["G"] * _points(case)
    if case["op"] == "predictor_mx":
        return {"bytes": M * C * e + NO * nb * 17 + (NO * 4 if case["bias"] else 0) + M * NO * e,
                "flops": 2 * M * C * NO}
    return {"bytes": M * C * e + NO * C * e + M * NO * 4 + M * C * 4 + NO * C * 4 + (NO * 4 if case["bias"] else 0),
            "flops": 4 * M * C * NO}


# ------------------------------------------------------- 64-bit definition ---

def _exact_mx(x):
    """Values (fp64 [M, C]) and scale exponents of the format's definition: 2^e with
    e = floor(log2(largest magnitude)) - 2 (at least -127), elements rounded to the
    nearest multiple of their binade's step (half a unit below 2), ties to even, at most 6."""
    M, C = x.shape
    nb = (C + 31) // 32
    v = torch.cat((x.double(), torch.zeros(M, nb * 32 - C, dtype=torch.float64, device=x.device)), dim=1)
    v = v.reshape(M, nb, 32)
    amax = v.abs().max(dim=2).values
    e = torch.where(amax > 0, torch.frexp(amax).exponent.long() - 3, torch.full_like(amax, -127, dtype=torch.long))
    e = torch.clamp(e, min=-127).unsqueeze(2)
    q = torch.ldexp(v, -e)
    step = torch.ldexp(torch.ones_like(q), torch.clamp(torch.frexp(q).exponent.long() - 2, min=-1))
    q = torch.clamp(torch.round(q / step) * step, -6.0, 6.0)
    return torch.ldexp(q, e).reshape(M, nb * 32)[:, :C], e.squeeze(2) + 127


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "mx":
        values, scale = _exact_mx(state["x"])
        return values, scale.to(torch.uint8)
    if op == "orthogonalize":
        a, b, c = COEFFICIENTS
        x = state["x"].double()
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
        for _ in range(STEPS):
            # the smaller side's Gram matrix; the other side gives the same product
            if x.shape[1] <= x.shape[2]:
                s = x @ x.mT
                x = a * x + b * (s @ x) + c * (s @ (s @ x))
            else:
                s = x.mT @ x
                x = a * x + b * (x @ s) + c * ((x @ s) @ s)
        return x
    G, P = case["G"], _points(case)
    # record slot of each projection channel
    slot = [(o // (2 * P)) * 3 * P + o % (2 * P) if o < 2 * G * P
            else ((o - 2 * G * P) // P) * 3 * P + 2 * P + (o - 2 * G * P) % P for o in range(3 * G * P)]
    slot = torch.tensor(slot, device="cuda")
    if op == "predictor_mx":
        low, high = (state["codes"] & 15).long(), (state["codes"] >> 4).long()
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
        w = torch.empty(low.shape[0], 2 * low.shape[1], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[low], table[high]
        w = torch.ldexp(w, (state["scales"].long() - 127).repeat_interleave(32, dim=1))[:, :case["C"]]
        q, _ = _exact_mx(state["y"])
        params = q @ w.mT
        if state["bias"] is not None:
            params += state["bias"].double()
        records = torch.empty_like(params)
        records[:, slot] = params
        return records.view(-1, G, 3 * P)
    gp = state["grad_offset_mask"].double().view(-1, 3 * G * P)[:, slot]
    out = [gp @ state["weight"].double(), gp.mT @ state["y"].double()]
    return out + ([gp.sum(dim=0)] if case["bias"] else [])
