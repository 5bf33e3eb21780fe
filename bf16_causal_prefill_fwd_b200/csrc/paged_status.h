// The paged-cache kernels' device status word, for b200attn_check (which has
// synchronised): returns it and clears it, or B200ATTN_ERR_CUDA.
#pragma once
int b200_paged_take_status();
