// mx4_launch.h -- launchers of the microscaled 4-bit operators and of the routing to experts.  The ABI layer (api.cu) has
// checked every argument.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace qmm {

constexpr int kMoeMaxExperts = 1024;   // one a thread of the block that sorts
constexpr int kMoeMaxK = 32;           // one a lane

struct Mx4QuantArgs {
  const void *x;
  int64_t x_matrix, x_row;         // strides in elements
  const int32_t *places;           // [rows, k], or null: row r stays row r
  void *codes, *scales;
  int64_t matrices, rows, K;
  int64_t k, out_rows;             // of places
  bool bf16, sorted;               // sorted: x has out_rows rows, and each place's row stays there
};
cudaError_t launch_mx4_quantize(const Mx4QuantArgs &a, cudaStream_t s);
cudaError_t launch_mx4_dequant(const void *codes, const void *scales, float *w, int64_t matrices, int64_t rows, int64_t K,
                               cudaStream_t s);

struct Mx4GemmArgs {
  const void *x_codes, *x_scales, *codes, *scales;
  const int32_t *starts, *counts;  // [experts], or null: all M rows go to the one matrix
  void *y;
  int64_t M, N, K, experts;
  int64_t routed;                  // rows of all experts together, about
  bool bf16, gated;
};
// Tokens of a tile of such a call (+ 1024: of a pair of CTAs).
int mx4_gemm_tile(const Mx4GemmArgs &a);
cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, cudaStream_t s);
cudaError_t read_clear_mx4_status(int *status, cudaStream_t s);
void set_mx4_test_wait(unsigned long long limit_ns);

struct MoePlanArgs {
  const void *logits;
  int64_t stride, T, E, k;
  bool bf16, normalize;
  int32_t *experts;
  float *weights;
  int32_t *places, *starts, *counts;
};
cudaError_t launch_moe_plan(const MoePlanArgs &a, cudaStream_t s);

struct MoeCombineArgs {
  const void *y;
  const float *weights;            // null: all 1
  const int32_t *places;
  void *out;
  int64_t T, k, R, N;
  bool y_bf16, out_bf16;
};
cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t s);

}  // namespace qmm
