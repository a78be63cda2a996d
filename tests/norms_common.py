"""The norms around a block in 64 bits, with the size of each result's terms: what its error in
fp32 arithmetic is a multiple of.

Counted with u = 2^-24, for the kernels' sums of at most 16 elements a thread and two trees of
five (26 additions): r_post and r_pre are off by 13 u of a sum of squares, 3 u of the root and
half of what their elements are off by. Then, relative to the sizes below,
  y     20 u of r_post, 10 u of the sigmoid (and |z| u where 2^x is approximate), 4 products: 40 u
  yh, u another 40 u, with RHO = rms of y's terms / rms of y: what cancels in y shows in r_pre
  dY    the mean of e yh: 26 u and its factors' 40 u; with yh's and r_pre's own: 150 u
  f     15 u more; dgate 35 more, db the second mean and its factors: 270 u
and a column's sum over T rows adds at most T u."""
import torch


def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def forward(x, b, post, pre, gate, scale, eps, post_norm=True, pre_norm=True):
    """dict of y, u, r_post, r_pre and of sizes Y, U, and yh's, bh, g, h = 1 - g."""
    x = x.double()
    d = x.shape[-1]
    one = torch.ones(d, dtype=torch.float64)
    o = {"pre": one if pre is None else pre.double(), "post": one if post is None else post.double()}
    o["g"], o["h"] = torch.ones(()).double(), torch.zeros(()).double()
    if gate is not None:
        z = gate.double() if gate.dim() == x.dim() else gate.double().unsqueeze(-1)
        o["g"], o["h"] = sigmoid(z), sigmoid(-z)
    o["bh"] = torch.zeros_like(x)
    o["y"], o["Y"] = x, x.abs()
    if b is not None:
        b = b.double()
        o["r_post"] = 1 / torch.sqrt((b * b).mean(-1, keepdim=True) + eps) if post_norm else torch.ones(()).double()
        o["bh"] = b * o["r_post"]
        n = o["g"] * o["bh"] * o["post"]
        o["y"], o["Y"] = scale * x + n, abs(scale) * x.abs() + n.abs()
    if pre_norm:
        ms = (o["y"] ** 2).mean(-1, keepdim=True) + eps
        o["r_pre"] = 1 / torch.sqrt(ms)
        o["rho"] = torch.sqrt(((o["Y"] ** 2).mean(-1, keepdim=True) + eps) / ms) + 1
        o["yh"] = o["y"] * o["r_pre"]
        o["Yh"] = o["r_pre"] * (o["Y"] + o["y"].abs() * o["rho"])
        o["u"], o["U"] = o["pre"] * o["yh"], o["pre"].abs() * o["Yh"]
    return o


def backward(dy, du, x, b, post, pre, gate, scale, eps, post_norm=True, pre_norm=True):
    """{name: (value, size)} of dx, db, dgate, dpost, dpre."""
    o = forward(x, b, post, pre, gate, scale, eps, post_norm, pre_norm)
    dY = torch.zeros_like(o["y"]) if dy is None else dy.double()
    D = dY.abs()
    out = {}
    if pre_norm:
        du = du.double()
        e = o["pre"] * du
        dY = dY + o["r_pre"] * (e - o["yh"] * (e * o["yh"]).mean(-1, keepdim=True))
        D = D + o["r_pre"] * o["rho"] * (e.abs() + o["Yh"] * (e.abs() * o["Yh"]).mean(-1, keepdim=True))
        out["dpre"] = ((du * o["yh"]).flatten(0, -2).sum(0), (du.abs() * o["Yh"]).flatten(0, -2).sum(0))
    if b is None:
        out["dx"] = (dY, D)
        return out
    out["dx"] = (scale * dY, abs(scale) * D)
    f, F, bh = o["g"] * dY * o["post"], (o["g"] * o["post"]).abs() * D, o["bh"]
    fb, Fb = f * bh, F * bh.abs()
    r = o["r_post"]
    if post_norm:
        out["db"] = (r * (f - bh * fb.mean(-1, keepdim=True)), r * (F + bh.abs() * Fb.mean(-1, keepdim=True)))
    else:
        out["db"] = (f, F)
    if gate is not None:
        out["dgate"] = (o["h"] * fb, o["h"] * Fb)
        if gate.dim() < x.dim():
            out["dgate"] = tuple(v.sum(-1) for v in out["dgate"])
        else:
            # for 16-bit results 2^x flushes what is under 2^-126: 1 - g is off by that much at
            # most, which is 2^-102 in units of 2^-24
            out["dgate"] = (out["dgate"][0], out["dgate"][1] + 2.0 ** -102 * Fb / C["dgate"])
    out["dpost"] = ((o["g"] * dY * bh).flatten(0, -2).sum(0), (o["g"] * D * bh.abs()).flatten(0, -2).sum(0))
    return out


# multiples of 2^-24 (docstring): of the forward's results and the gradients'
C = {"y": 40, "u": 80, "dx": 155, "db": 270, "dgate": 230, "dpost": 200, "dpre": 60}
