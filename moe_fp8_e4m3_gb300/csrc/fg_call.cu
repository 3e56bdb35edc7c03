// fg_call.cu - calls of a serving step with their arguments in one record.
#include <cstdint>
#include <cstring>

#include "fg.h"

namespace {

struct Words {
    const unsigned char* p;
    int64_t word(int i) const {
        int64_t v;
        std::memcpy(&v, p + 8 * i, 8);
        return v;
    }
    // an integer that does not fit the entry point's type becomes one that every entry point refuses
    int i32(int i) const {
        const int64_t v = word(i);
        return v == static_cast<int>(v) ? static_cast<int>(v) : -1;
    }
    float f32(int i) const {
        double v;
        std::memcpy(&v, p + 8 * i, 8);
        return static_cast<float>(v);
    }
    template <class T>
    T* ptr(int i) const { return reinterpret_cast<T*>(static_cast<uintptr_t>(word(i))); }
    fg_stream_t stream(int i) const { return ptr<CUstream_st>(i); }
};

}  // namespace

extern "C" int fg_call(int id, const void* words) {
    if (!words) return FG_ERR_INVALID_ARG;
    const Words w{static_cast<const unsigned char*>(words)};
    using C32 = const int32_t;
    using I32 = int32_t;
    using U8 = uint8_t;
    using CU8 = const uint8_t;
    switch (id) {
        case FG_CALL_BUILD_BLOCK_TABLES:
            return fg_build_block_tables(w.i32(0), w.i32(1), w.i32(2), w.i32(3), w.i32(4), w.i32(5), w.ptr<C32>(6), w.ptr<C32>(7),
                                         w.ptr<I32>(8), w.ptr<C32>(9), w.ptr<I32>(10), w.ptr<I32>(11), w.ptr<I32>(12),
                                         w.ptr<I32>(13), w.ptr<I32>(14), w.ptr<I32>(15), w.stream(16));
        case FG_CALL_QK_NORM_ROPE:
            return fg_qk_norm_rope(w.i32(0), w.i32(1), w.i32(2), w.i32(3), w.i32(4), w.i32(5), w.ptr<const void>(6), w.word(7),
                                   w.ptr<const void>(8), w.word(9), w.ptr<const void>(10), w.ptr<const void>(11), w.f32(12),
                                   w.ptr<C32>(13), w.ptr<const float>(14), w.i32(15), w.ptr<void>(16), w.word(17),
                                   w.ptr<void>(18), w.word(19), w.stream(20));
        case FG_CALL_KV_APPEND_MXFP4:
            return fg_kv_append_mxfp4(w.i32(0), w.i32(1), w.i32(2), w.i32(3), w.i32(4), w.ptr<const void>(5), w.word(6),
                                      w.ptr<const void>(7), w.word(8), w.ptr<C32>(9), w.ptr<U8>(10), w.ptr<U8>(11),
                                      w.ptr<U8>(12), w.ptr<U8>(13), w.stream(14));
        case FG_CALL_KV_GATHER_MXFP4:
            return fg_kv_gather_mxfp4(w.i32(0), w.i32(1), w.i32(2), w.i32(3), w.i32(4), w.ptr<C32>(5), w.ptr<CU8>(6),
                                      w.ptr<CU8>(7), w.ptr<CU8>(8), w.ptr<CU8>(9), w.ptr<void>(10), w.word(11),
                                      w.ptr<void>(12), w.word(13), w.stream(14));
        case FG_CALL_PAGED_ATTENTION_MXFP4:
            return fg_paged_attention_mxfp4(w.i32(0), w.i32(1), w.i32(2), w.i32(3), w.i32(4), w.i32(5), w.i32(6), w.i32(7),
                                            w.ptr<const void>(8), w.ptr<CU8>(9), w.ptr<CU8>(10), w.ptr<CU8>(11), w.ptr<CU8>(12),
                                            w.ptr<C32>(13), w.ptr<C32>(14), w.ptr<C32>(15), w.f32(16), w.i32(17),
                                            w.ptr<void>(18), w.ptr<void>(19), w.stream(20));
        default:
            return FG_ERR_INVALID_ARG;
    }
}
