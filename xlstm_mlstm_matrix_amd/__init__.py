"""mLSTM cell forward (xLSTM) on AMD MI355X (gfx950).

The compute path is the HIP library ``libmlstm.so`` behind the C ABI in
``include/mlstm.h`` and ``include/mlstm_ops.h``; :mod:`.binding` marshals torch
tensors into it.
"""
from .binding import (BF16, F32, MlstmError, deltarule_bwd, deltarule_fwd, deltarule_step,  # noqa: F401
                      fwd_chunkwise, groupnorm_bwd, groupnorm_fwd, lib, linattn_bwd, linattn_fwd, linattn_step,
                      qknorm_bwd, qknorm_fwd, rope_frequencies, status_string, step, workspace_size)

__version__ = "0.1.0"
