"""A regularised residual DLRM training step: the tower operators next to the embedding core.

    pooled  = emb_bag_fwd(tables, bags)                       [B, F, D]
    normed  = group norm of each sample's pooled vectors over its F tables, in groups of D
    vectors = dropout(normed)                                 (feature dropout)
    inter   = dot interaction of the bottom MLP's output with them
    h_0     = dropout(gelu(inter W_0 + b_0))
    h_i     = h_{i-1} + dropout(gelu(h_{i-1} W_i + b_i))      (residual blocks)
    logit   = h_last w + b,  logistic loss

and the backward of all of it: one dense_bwd per layer (the skip connection's gradient added and
the activation and dropout of the layer below undone in its epilogue), the interaction's, the
group norm's, and SGD on the dense parameters, the norm's scale and shift and the embedding rows.
The dropout masks are drawn from (seed, layer, step counter on the device), so nothing is stored
for them and a captured step draws new masks at every replay.

    python -m embedding_lookup_feature_amd.residual --steps 20
"""
import argparse

import torch

from . import dlrm, synth, tower
from . import embcore as ec


class ResidualDLRMStep(dlrm.DLRMStep):
    """Buffers and parameters for one workload; `train_step` runs one SGD step."""

    def __init__(self, wl: synth.Workload, tables: ec.Tables, device, width: int = 1024, blocks: int = 2,
                 groups: int = 8, p: float = 0.1, p_features: float = 0.05, seed: int = 1234):
        super().__init__(wl, tables, device, top=(width,) * (1 + blocks) + (1,))
        dt, B, D, F = self.dtype, wl.batch, wl.dim, wl.num_tables
        e = lambda *s: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device=device)  # noqa: E731
        self.groups = groups
        self.normed, self.vectors, self.dnormed = e(B * F, D), e(B * F, D), e(B * F, D)
        self.mean, self.rstd = f32(B, groups), f32(B, groups)
        self.gn = torch.cat([torch.ones(D), torch.zeros(D)]).to(device)  # gamma, beta
        self.dgn = f32(2 * D)
        self.pre = [e(B, width) for _ in range(1 + blocks)]
        self.dh, self.dz = [e(B, width) for _ in range(2)], [e(B, width) for _ in range(2)]
        self.step = torch.zeros(1, dtype=torch.int64, device=device)
        # one offset per layer, far enough apart for every step to have masks of its own
        self.drops = [tower.Dropout(p, seed, (i + 1) << 48, self.step) for i in range(1 + blocks)]
        self.drop_features = tower.Dropout(p_features, seed, 0, self.step)
        need = [self.lin_ws.numel(), tower.group_norm_fwd_workspace_bytes(B, F, D, groups),
                tower.group_norm_bwd_workspace_bytes(B, F, D, groups)]
        for N, K in self.top.shapes:
            need += [tower.dense_fwd_workspace_bytes(B, K, N), tower.dense_bwd_workspace_bytes(B, K, N)]
        self.lin_ws = torch.empty(max(need), dtype=torch.uint8, device=device)

    @property
    def gamma(self):
        return self.gn[: self.wl.dim]

    @property
    def beta(self):
        return self.gn[self.wl.dim:]

    def _rows(self, t):
        return t.view(self.wl.batch * self.wl.num_tables, self.wl.dim)

    def forward(self, dense, bags, train: bool = True):
        """Logits [B, 1]; without `train`, no dropout and nothing kept for a backward."""
        F, ws = self.wl.num_tables, self.lin_ws
        h = dense
        for i, (w, b) in enumerate(zip(self.bottom.w, self.bottom.b)):
            ec.linear_fwd(h, w, b, self.h_bot[i], relu=True)
            h = self.h_bot[i]
        ec.emb_bag_fwd(self.tables, bags, self.emb)
        tower.group_norm_fwd(self._rows(self.emb), self.gamma, self.beta, self.normed, self.mean, self.rstd, positions=F,
                             groups=self.groups, workspace=ws)
        vectors = self.normed
        if train:
            vectors = tower.act_dropout_fwd(self.normed, self.vectors, dropout=self.drop_features)
        ec.dot_interact_fwd(self.h_bot[-1], vectors.view_as(self.emb), self.inter)
        h = self.inter
        for i in range(len(self.pre)):
            tower.dense_fwd(h, self.top.w[i], self.top.b[i], self.h_top[i], act="gelu",
                            dropout=self.drops[i] if train else None, residual=h if i > 0 else None,
                            pre=self.pre[i] if train else None, workspace=ws)
            h = self.h_top[i]
        ec.linear_fwd(h, self.top.w[-1], self.top.b[-1], self.h_top[-1], relu=False)
        return self.h_top[-1]

    def backward(self, dense, labels):
        """Loss and every gradient, after forward(train=True)."""
        F, ws, n = self.wl.num_tables, self.lin_ws, len(self.pre)
        ec.bce_logits(self.h_top[-1], labels, self.loss, self.dlogit, workspace=ws)
        dh, dz = self.dh[0], self.dz[0]  # gradients of the residual stream and of the pre-activation
        ec.linear_bwd(self.h_top[n - 1], self.top.w[n], self.dlogit, self.top.dw[n], self.top.db[n], dx=dh, workspace=ws)
        tower.act_dropout_bwd(dh, self.pre[n - 1], dz, act="gelu", dropout=self.drops[n - 1])
        for i in reversed(range(1, n)):
            below_h, below_z = self.dh[(n - i) % 2], self.dz[(n - i) % 2]
            tower.dense_bwd(self.h_top[i - 1], self.top.w[i], dz, self.top.dw[i], self.top.db[i], dx=below_h, dres=dh,
                            dzb=below_z, pre=self.pre[i - 1], act="gelu", dropout=self.drops[i - 1], workspace=ws)
            dh, dz = below_h, below_z
        tower.dense_bwd(self.inter, self.top.w[0], dz, self.top.dw[0], self.top.db[0], dx=self.dout, workspace=ws)
        ec.dot_interact_bwd(self.h_bot[-1], self.vectors.view_as(self.emb), self.dout, self.dx0, self.demb)
        tower.act_dropout_bwd(self._rows(self.demb), None, self.dnormed, dropout=self.drop_features)
        tower.group_norm_bwd(self.dnormed, self._rows(self.emb), self.gamma, self.beta, self.mean, self.rstd,
                             self._rows(self.demb), self.dgn[: self.wl.dim], self.dgn[self.wl.dim:], positions=F,
                             groups=self.groups, workspace=ws)
        dz = self._g(0, self.wl.dim)
        ec.relu_bwd(self.dx0, self.h_bot[-1], dz)
        for i in reversed(range(len(self.bottom.w))):
            x = self.h_bot[i - 1] if i > 0 else dense
            dx = self._g((len(self.bottom.w) - i) % 2, x.shape[1]) if i > 0 else None
            ec.linear_bwd(x, self.bottom.w[i], dz, self.bottom.dw[i], self.bottom.db[i], dx=dx, relu_mask=(i > 0),
                          workspace=ws)
            dz = dx

    def train_step(self, dense, bags, labels, emb_ws):
        """Forward, backward and SGD on everything; the step counter then moves the masks on."""
        lr = self.wl.lr
        ec.emb_grad_prepare(self.tables, bags, emb_ws)
        self.forward(dense, bags)
        self.backward(dense, labels)
        self.bottom.sgd(lr)
        self.top.sgd(lr)
        ec.sgd_dense(self.gn, self.dgn, lr)
        ec.emb_grad_apply(self.tables, bags, self.demb, lr, emb_ws)
        self.step += 1


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--batch", type=int, default=4096)
    ap.add_argument("--rows", type=int, default=20_000, help="rows of each of the 26 tables")
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--dropout", type=float, default=0.1)
    ap.add_argument("--lr", type=float, default=0.001)
    args = ap.parse_args(argv)
    dev = "cuda"
    wl = synth.WORKLOADS["train_step"].scaled(name="residual", batch=args.batch, rows=(args.rows,) * 26,
                                               lr=args.lr)
    W, ro = synth.make_tables(wl, dev)
    idx, off = synth.make_indices(wl, dev)
    tables, bags = ec.Tables(W, ro), ec.Bags(idx, off, wl.batch)
    model = ResidualDLRMStep(wl, tables, dev, blocks=args.blocks, p=args.dropout)
    dense = synth.make_dense(wl, dev, k_pad=model.k_pad)
    labels = synth.make_labels(wl, dev)
    emb_ws = ec.alloc_workspace(tables, bags)
    for s in range(args.steps):
        model.train_step(dense, bags, labels, emb_ws)
        if s % 5 == 0 or s == args.steps - 1:
            print(f"step {s}: loss {float(model.loss):.5f}", flush=True)


if __name__ == "__main__":
    main()
