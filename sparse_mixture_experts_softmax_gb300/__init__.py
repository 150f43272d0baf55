"""GB300-native (sm_103a) sparse top-k mixture-of-experts training step.

The layer lives in the CUDA library ``libmoe_gb300.so`` behind the C ABI of
``include/moe.h``; ``binding`` is its thin ctypes binding and ``layer`` a small
helper that owns the device buffers of one layer.  ``norm`` is the layer norm of
the residual block around it, ``decode`` the layer for a few tokens
(``include/moe_block.h``) and ``block`` the three together.
"""

from .binding import (MoEError, make_config, make_grads, make_norm_config,  # noqa: F401
                      make_params, make_weights,
                      moe_backward, moe_decode, moe_decode_init, moe_decode_status,
                      moe_decode_workspace_size, moe_device_status, moe_dispatch_noalloc,
                      moe_forward,
                      moe_get_hidden, moe_get_intermediates, moe_get_routing, moe_grouped_gemm,
                      moe_host_staging_size, moe_last_launch_count, moe_norm_backward,
                      moe_norm_forward, moe_norm_workspace_size, moe_status_string,
                      moe_train_step, moe_train_step_host, moe_train_steps_host,
                      moe_workspace_size)
