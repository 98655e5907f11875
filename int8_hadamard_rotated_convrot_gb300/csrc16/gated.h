// Launch interface between the C-ABI layer (api_gated.cu) and the kernels of the
// gated feed-forward's projections (include/convrot_block.h). Arguments are
// validated; operands have rows that start on 16 bytes.
#pragma once

#include "../csrc/block.h"

namespace convrot {

// y (and gate, up): many rows, and few.
cudaError_t launch_gated_gemm(const convrot_gated_linear_args &a, cudaStream_t stream);
bool gated_few_takes(int64_t m, int64_t n, int64_t k);
cudaError_t launch_gated_few(const convrot_gated_linear_args &a, cudaStream_t stream);

// dx = dg w_gate + du w_up (partial: gated_dx_partial_bytes) and dw = dg^T x, du^T x from dg and du [m, ldd].
int64_t gated_dx_partial_bytes(int64_t m, int64_t n, int64_t k);
cudaError_t launch_gated_dx(const convrot_gated_linear_backward_args &a, const void *dg, const void *du, int64_t ldd, float *partial, cudaStream_t stream);
cudaError_t launch_gated_dw(const convrot_gated_linear_backward_args &a, const void *dg, const void *du, int64_t ldd, cudaStream_t stream);

// dg and du [m, ldd] (ldd a multiple of 8; columns past n become zero) and, where partial is not null, the column sums:
// partial holds gated_grad_chunks(m, n) x 2 x n floats.
int64_t gated_grad_chunks(int64_t m, int64_t n);
cudaError_t launch_gated_grad(const convrot_gated_linear_backward_args &a, void *dg, void *du, int64_t ldd, float *partial, cudaStream_t stream);

// A copy [rows, ldo] (ldo a multiple of 8, 16-byte aligned) of 16-bit elements with rows that start anywhere.
cudaError_t launch_align_rows(const void *x, int64_t rows, int64_t cols, int64_t ld, void *out, int64_t ldo, cudaStream_t stream);

// Shared memory and tensor-memory columns of every launch form, for the check that no mix of blocks waits for columns.
int gated_gemm_shared(int form, int *columns);  // 0 past the last form
int gated_few_shared(int form, int *columns);

}  // namespace convrot
