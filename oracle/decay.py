"""float64 oracle of decay attention: the recurrence with one constant decay per head.

TEST INFRASTRUCTURE ONLY (never imported by the product path).

Token by token, in numpy float64, for one sequence of all heads ([H,T,d], states
[H,dk,dv]), with lambda_h = exp(ld[h]):

    S_t = lambda_h S_{t-1} + k_t^T v_t ,     o_t = q_t S_t ,

and its adjoint R_t = dL/dS_t = lambda_h R_{t+1} + q_t^T do_t with R_T += dS_T:

    dq_t = do_t S_t^T ,  dk_t = v_t R_t^T ,  dv_t = k_t R_t ,  dS_0 = lambda_h R_1 .
"""
from __future__ import annotations

import numpy as np


def _lam(ld):
    return np.exp(np.asarray(ld, np.float64))[:, None, None]


def fwd(q, k, v, ld, s0=None):
    """(o [H,T,dv], S_T [H,dk,dv]); T may be zero."""
    H, T, dk = q.shape
    dv = v.shape[-1]
    lam = _lam(ld)
    S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0, np.float64)
    o = np.zeros((H, T, dv))
    for t in range(T):
        S = lam * S + k[:, t, :, None] * v[:, t, None, :]
        o[:, t] = np.einsum("hk,hkv->hv", q[:, t], S)
    return o, S


def bwd(q, k, v, ld, do, s0=None, ds=None):
    """(dq, dk, dv, dS_0) of one sequence."""
    H, T, dk_ = q.shape
    dv_ = v.shape[-1]
    lam = _lam(ld)
    S = np.zeros((H, dk_, dv_)) if s0 is None else np.array(s0, np.float64)
    R = np.zeros((H, dk_, dv_)) if ds is None else np.array(ds, np.float64)
    dq, dk, dv = np.zeros((H, T, dk_)), np.zeros((H, T, dk_)), np.zeros((H, T, dv_))
    for t in range(T):
        S = lam * S + k[:, t, :, None] * v[:, t, None, :]
        dq[:, t] = np.einsum("hv,hkv->hk", do[:, t], S)
    for t in reversed(range(T)):
        R = R + q[:, t, :, None] * do[:, t, None, :]
        dk[:, t] = np.einsum("hv,hkv->hk", v[:, t], R)
        dv[:, t] = np.einsum("hk,hkv->hv", k[:, t], R)
        R = lam * R
    return dq, dk, dv, R
