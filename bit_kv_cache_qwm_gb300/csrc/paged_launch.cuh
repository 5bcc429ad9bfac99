// Launchers of the paged caches' kernels that take their call's arguments
// (each returns cudaGetLastError() of its launch; the arguments are checked).
#pragma once

#include "qwm_internal.cuh"

namespace qwm {
namespace paged {

cudaError_t launch_plan(const qwm_paged_plan_args& a, int shift, cudaStream_t st);
cudaError_t launch_release(const qwm_paged_release_args& a, int shift, cudaStream_t st);
cudaError_t launch_append(const qwm_paged_append_args& a, int shift, cudaStream_t st);
cudaError_t launch_append8(const qwm_paged8_append_args& a, int shift, cudaStream_t st);
cudaError_t launch_read8(const qwm_paged8_read_args& a, int shift, cudaStream_t st);
cudaError_t launch_bounds8(const qwm_paged8_bounds_args& a, int shift, cudaStream_t st);
cudaError_t launch_select8(const qwm_paged8_select_args& a, int shift, cudaStream_t st);
cudaError_t launch_qk_norm_rope(const qwm_qk_norm_rope_args& a, cudaStream_t st);

}  // namespace paged
}  // namespace qwm
