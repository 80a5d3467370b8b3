"""Softmax cross entropy of alpha*X*W^T and its gradients in 64 bits, from the
formulas (numpy): the plain implementation that the kernels are tested
against."""
import numpy as np

IGNORE = -100


def forward(x, w, labels, alpha=1.0):
    """z, loss, lse (0 where the label is IGNORE)."""
    keep = labels != IGNORE
    z = alpha * (np.where(keep[:, None], x, 0.0) @ w.T)
    m = z.max(1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(1))
    loss = lse - z[np.arange(len(labels)), np.where(keep, labels, 0)]
    return z, np.where(keep, loss, 0.0), np.where(keep, lse, 0.0)


def dlogits(z, labels, lse, dloss, dlse=None):
    """The gradient of z (zero rows where the label is IGNORE)."""
    keep = labels != IGNORE
    q = np.where(keep, dloss, 0.0)
    p = q if dlse is None else q + np.where(keep, dlse, 0.0)
    dz = p[:, None] * np.exp(np.where(keep[:, None], z - lse[:, None], -np.inf))
    rows = np.flatnonzero(keep)
    dz[rows, labels[rows]] -= q[rows]
    return dz


def gradients(x, w, labels, dz, alpha=1.0):
    x = np.where((labels != IGNORE)[:, None], x, 0.0)
    return alpha * (dz @ w), alpha * (dz.T @ x)
