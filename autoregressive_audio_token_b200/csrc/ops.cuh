// ops.cuh -- what the translation units of the serving operators share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

namespace m3 {

// The thread-local message behind m3_last_error (m3.cu).
int set_error(int code, const std::string& msg);

// log2 of a page size the operators take (a power of two, 16..1024), or -1.
int page_shift(int page);

// SMs of the current device.
int sm_count();

// m3_attn_prompt (include/m3_ops.h) with the error word its waits report to
// (null: the one m3_ops_sync_status reads).
int attn_prompt(int dtype, int n_seq, int n_q, int n_k, int Hq, int Hkv, int D, const void* q,
                int64_t q_token, int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                const void* v, int64_t v_token, int64_t v_head, const int32_t* cu_q,
                const int32_t* cu_k, float scale, void* out, int64_t o_token, int64_t o_head,
                float* lse, int* err, void* cuda_stream);

}  // namespace m3
