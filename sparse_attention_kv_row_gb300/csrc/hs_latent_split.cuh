// hs_latent_split.cuh -- the tensor-core kernels of latent attention (16-bit types,
// 512 + 64 dims), as the entry point calls them.
#pragma once

#include "hs_latent.cuh"

namespace hs {

// hs_latent_split.cu: few query rows a token.
int64_t latent_split_workspace(int in_dtype, bool codes, const DeviceInfo& dev);
bool latent_split_fits(const LatentParams& p);
hs_err latent_split_launch(const LatentParams& p, int in_dtype, bool codes, void* workspace,
                           const DeviceInfo& dev, cudaStream_t stream);

}  // namespace hs
