// What the C entry points' files share: the last error's text, status results, workspace checks and layouts.
#pragma once

#include <stdint.h>

#include <string>

#include "../../include/kda.h"
#include "kda_layer.cuh"

namespace kda {

void set_last_error(const char* msg);

namespace api {

constexpr size_t ALIGN = 256;
inline size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }

inline kda_status fail(kda_status st, const char* msg) {
    set_last_error(msg);
    return st;
}
inline kda_status cuda_result(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return KDA_OK;
    set_last_error((std::string(where) + ": " + cudaGetErrorString(e)).c_str());
    return KDA_ERR_CUDA;
}
inline kda_status check_ws(const void* ws, size_t bytes, size_t need, const char* what) {
    if (need == 0) return KDA_OK;
    if (ws && reinterpret_cast<uintptr_t>(ws) % ALIGN == 0 && bytes >= need) return KDA_OK;
    set_last_error((std::string(what) + " missing, not 256-byte aligned or below " + std::to_string(need) + " bytes").c_str());
    return KDA_ERR_WORKSPACE;
}

inline int esize(kda_dtype io) { return io == KDA_BF16 ? 2 : 4; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The token axis of B sequences of T tokens, or of N packed ones.
inline kda_status make_axis(int B, int T, int N, const int32_t* cu, int D, kda_dtype io, TokenAxis& ax) {
    if (B < 1 || T < 0 || D < 1) return fail(KDA_ERR_INVALID_ARG, "B and D must be >= 1 and T >= 0");
    if (io != KDA_BF16 && io != KDA_FP32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if ((long long)B * T > (1LL << 30)) return fail(KDA_ERR_UNSUPPORTED, "too many tokens");
    if (D > (1 << 20)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^20 channels");
    if (cu) {
        if (B != 1) return fail(KDA_ERR_INVALID_ARG, "packed sequences need B == 1");
        if (N < 1) return fail(KDA_ERR_INVALID_ARG, "packed sequences need N >= 1");
    }
    ax = {cu, cu ? N : B, B, T};
    return KDA_OK;
}

struct Carver {
    char* p;
    size_t used = 0;
    template <class T>
    T* take(size_t bytes) {
        T* r = reinterpret_cast<T*>(p + used);
        used += bytes;
        return bytes ? r : nullptr;
    }
};

}  // namespace api
}  // namespace kda
