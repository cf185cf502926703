// Host-side declarations of the mixture-of-experts layer (moe_layer.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tail {

struct MoeLayerArgs;

struct MoeLayerPlan {
  bool ok;
  int format;   // Format of moe_layer.cu
  int G;        // tokens of one expert that share a pass over its weights
  int columns;  // n-tiles of the kernel's form: 1, 2 or 4
  int R;        // activation rows in shared memory
  int all_rows; // every token's rows of the first product stay there
  int smem;     // dynamic shared memory of the expert kernels
  int grid;
  int ksplit1, ksplit2;  // warps that split the columns of W1's and W2's rows
};

MoeLayerPlan plan_moe_layer(int T, int topk, int nsh, int E, int H, int I, int N1, bool fp4, int max_smem, int num_sms);
cudaError_t launch_moe_layer(const MoeLayerArgs& a, const MoeLayerPlan& p, cudaStream_t stream);

}  // namespace tail
