"""Gaussians predicted from the tokens of image patches, trained through the rasterizer.

Every patch of a scene's context images is a token. Blocks of attention and a feed-forward
part mix the tokens of a scene, and each token becomes one Gaussian on its patch's ray. The
scene is then rendered from another camera, and the image's error is differentiated back
through the rasterizer and the token operators to the weights.

The scenes have different numbers of context images, so their tokens are packed into one row
and each token's keys are the span of its scene; the row's end is padding that sees nothing.
Queries and keys are normalised and rotated by their patch's place, the blocks' branches are
dropped out on their way into the residual stream, and so are whole Gaussians.

    python examples/predict_gaussians.py [steps]
"""
import math
import os
import sys

import numpy as np
import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gaussian_splatting_differentiable_amd as gsr  # noqa: E402
import scenegen  # noqa: E402
from gaussian_splatting_differentiable_amd import tokens  # noqa: E402

SIZE, PATCH, FOCAL = 64, 8, 64.0
GRID = SIZE // PATCH
WIDTH, HEADS, KV_HEADS, DIM, LAYERS = 256, 4, 2, 64, 2
DROP_BRANCH, DROP_GAUSSIAN = 0.1, 0.05


class Splat(torch.autograd.Function):
    """The rendered image of activated Gaussians (SH of degree 0)."""

    @staticmethod
    def forward(ctx, raster, means, log_scales, quats, opacities, sh):
        held = [t.detach().contiguous() for t in (means, log_scales, quats, opacities, sh)]
        raster.project(*held, 0)
        raster.run_frame(held[0].shape[0])
        ctx.raster = raster
        ctx.save_for_backward(*held)
        return raster.rgb.clone()

    @staticmethod
    def backward(ctx, d_rgb):
        raster, held = ctx.raster, ctx.saved_tensors
        raster.render_bwd(held[0].shape[0], d_rgb.contiguous())
        g = raster.project_bwd(*held, 0)
        return None, g["means"], g["log_scales"], g["quats"], g["opacities"], g["sh"]


class Draws:
    """Places in one stream of random numbers: every dropout of a run has its own."""

    def __init__(self, seed):
        self.seed, self.offset, self.on = seed, 0, True

    def drop(self, x, p, residual=None):
        if not self.on:
            return x if residual is None else x + residual
        at = self.offset
        self.offset += (x.numel() + 3) // 4  # a counter gives four draws
        return tokens.Dropout.apply(x, residual, p, self.seed, at, False)


def linear(x, weight):
    return F.linear(x, weight.to(x.dtype))


class Block(torch.nn.Module):
    def __init__(self):
        super().__init__()
        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols) / math.sqrt(cols))
        self.qkv = weight((HEADS + 2 * KV_HEADS) * DIM, WIDTH)
        self.out = weight(WIDTH, HEADS * DIM)
        self.up, self.down = weight(4 * WIDTH, WIDTH), weight(WIDTH, 4 * WIDTH)
        self.q_norm, self.k_norm = (torch.nn.Parameter(torch.ones(DIM)) for _ in range(2))

    def forward(self, x, spans, cos_sin, positions, draws):
        b, n, _ = x.shape
        # queries, keys and values stay views of the joint projection
        qkv = linear(F.layer_norm(x, (WIDTH,)), self.qkv).view(b, n, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), dim=2)
        q, k = tokens.QkNormRope.apply(q, k, self.q_norm, self.k_norm, cos_sin, positions,
                                       False, 1e-6)
        o = tokens.Attention.apply(q, k, v, spans, False, None)
        x = draws.drop(linear(o.reshape(b, n, HEADS * DIM), self.out), DROP_BRANCH, x)
        y = linear(F.gelu(linear(F.layer_norm(x, (WIDTH,)), self.up)), self.down)
        return draws.drop(y, DROP_BRANCH, x)


class Predictor(torch.nn.Module):
    """Patches [tokens][3 PATCH^2] to Gaussians in their cameras' frames."""

    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(WIDTH, 3 * PATCH * PATCH) / 14.0)
        self.blocks = torch.nn.ModuleList(Block() for _ in range(LAYERS))
        self.head = torch.nn.Parameter(torch.randn(14, WIDTH) * 0.02)
        y, x = torch.meshgrid(torch.arange(GRID), torch.arange(GRID), indexing="ij")
        turn = 10.0 ** -torch.linspace(0, 2, DIM // 4)
        angle = torch.cat([place.reshape(-1, 1) * turn for place in (y, x)], 1)
        self.register_buffer("cos_sin", torch.cat([angle.cos(), angle.sin()], 1).contiguous())

    def forward(self, patches, rays, spans, positions, draws):
        x = linear(patches.bfloat16(), self.embed)[None]
        for block in self.blocks:
            x = block(x, spans, self.cos_sin, positions, draws)
        raw = linear(F.layer_norm(x, (WIDTH,)), self.head)[0].float()
        depth = 4.0 * torch.exp(0.5 * torch.tanh(raw[:, 0:1]))
        # a Gaussian about as wide as its patch at its depth, and where its ray is
        means = depth * (rays + 0.5 * PATCH / FOCAL * F.pad(torch.tanh(raw[:, 1:3]), (0, 1)))
        log_scales = torch.log(depth * PATCH / FOCAL) - 1.0 + torch.tanh(raw[:, 3:6])
        quats = F.normalize(raw[:, 6:10] + raw.new_tensor([1.0, 0.0, 0.0, 0.0]), dim=1)
        opacities = draws.drop(0.95 * torch.sigmoid(raw[:, 10]), DROP_GAUSSIAN)
        return means, log_scales, quats, opacities, raw[:, 11:14, None].transpose(1, 2)


def cameras(n):
    """n cameras beside each other that look the same way (x to the right)."""
    return [scenegen.pinhole(SIZE, SIZE, FOCAL, np.array([1, 0, 0, -0.3 * i, 0, 1, 0, 0,
                                                          0, 0, 1, 0], np.float32))
            for i in range(n)]


def render(scene, camera, device):
    held = [torch.from_numpy(np.ascontiguousarray(a)).to(device)
            for a in (scene.means, scene.log_scales, scene.quats, scene.opacities, scene.sh)]
    return Splat.apply(gsr.Rasterizer(camera, device=device, capacity=1 << 16), *held)


def make_data(device, views=(2, 1), pad=8):
    """Scenes of random Gaussians: the packed patches of `views` context images each, and
    one more image of each scene to be predicted."""
    patches, rays, at, spans, shift, goals = [], [], [], [], [], []
    px = (torch.arange(GRID) + 0.5) * PATCH
    y, x = torch.meshgrid(px, px, indexing="ij")
    ray = torch.stack([(x - SIZE / 2) / FOCAL, (y - SIZE / 2) / FOCAL, torch.ones_like(x)], -1)
    n = 0
    for i, count in enumerate(views):
        scene = scenegen.random_scene(50 + i, 300, SIZE, SIZE, FOCAL, depth=(3.0, 5.0),
                                      log_scale=(-2.0, 0.3), opacity=(1.5, 0.5))
        cams = cameras(count + 1)
        for j in range(count):
            image = render(scene, cams[j], device)
            p = image.view(3, GRID, PATCH, GRID, PATCH).permute(1, 3, 0, 2, 4)
            patches.append(p.reshape(GRID * GRID, -1))
            rays.append(ray.reshape(-1, 3))
            at.append(torch.arange(GRID * GRID, dtype=torch.int32))
            shift.append(torch.tensor([[0.3 * j, 0.0, 0.0]]).expand(GRID * GRID, 3))
        m = count * GRID * GRID
        spans += [[n, n + m]] * m
        goals.append((n, n + m, gsr.Rasterizer(cams[count], device=device, capacity=1 << 16),
                      render(scene, cams[count], device)))
        n += m
    patches.append(torch.zeros(pad, 3 * PATCH * PATCH, device=device))
    rays.append(torch.zeros(pad, 3))
    shift.append(torch.zeros(pad, 3))
    at.append(torch.zeros(pad, dtype=torch.int32))
    spans += [[0, 0]] * pad
    return dict(patches=torch.cat(patches), rays=torch.cat(rays).to(device),
                shift=torch.cat(shift).to(device), positions=torch.cat(at).to(device),
                spans=torch.tensor(spans, dtype=torch.int32, device=device), goals=goals)


def step(model, data, draws):
    """The mean squared error of the predicted scenes' images."""
    means, *rest = model(data["patches"], data["rays"], data["spans"], data["positions"], draws)
    means = means + data["shift"]  # from the context cameras' frames to the world
    loss = 0.0
    for lo, hi, raster, goal in data["goals"]:
        image = Splat.apply(raster, means[lo:hi], *(t[lo:hi] for t in rest))
        loss = loss + F.mse_loss(image, goal)
    return loss / len(data["goals"])


def train(steps=100, device="cuda", say=print):
    torch.manual_seed(0)
    model, draws = Predictor().to(device), Draws(seed=7)
    data = make_data(device)
    optimizer = torch.optim.Adam(model.parameters(), lr=5e-4)
    losses = []
    for i in range(steps):
        optimizer.zero_grad()
        loss = step(model, data, draws)
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
        if i % 20 == 0 or i == steps - 1:
            say(f"step {i}: mean squared error {losses[-1]:.4f}")
    draws.on = False
    with torch.no_grad():
        losses.append(float(step(model, data, draws)))
    say(f"without dropout: {losses[-1]:.4f}")
    return model, losses


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100)
