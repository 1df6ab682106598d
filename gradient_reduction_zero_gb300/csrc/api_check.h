// Checks of arguments that the entry points of lm_api.cpp, attn_api.cpp and
// tensors_api.cpp share: types, addresses, factors, and buffers of a call that
// overlap.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "api_util.h"

namespace dpz {

inline int check_elem_type(int dt, const char* what)
{
    if (dt != DPZ_F32 && dt != DPZ_BF16)
        return fail(DPZ_ERR_INVALID_ARG, "%s dtype %d is not supported", what, dt);
    return DPZ_OK;
}

inline int check_addr(const void* p, const char* what, size_t align)
{
    if (p == nullptr) return fail(DPZ_ERR_INVALID_ARG, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % align != 0)
        return fail(DPZ_ERR_ALIGN, "%s is not %d-byte aligned", what, (int)align);
    return DPZ_OK;
}

inline int check_ids(const void* p, int it, int64_t n, const char* what)
{
    if (it != DPZ_I32 && it != DPZ_I64)
        return fail(DPZ_ERR_INVALID_ARG, "%s id type %d is not supported", what, it);
    return n > 0 ? check_addr(p, what, it == DPZ_I32 ? 4 : 8) : DPZ_OK;
}

// A factor of the logits: beyond 1e30 the difference of two of them overflows.
inline int check_factor(float x, const char* what)
{
    if (!(x > 0.0f) || x > 1e30f)
        return fail(DPZ_ERR_INVALID_ARG, "%s = %g is outside (0, 1e30]", what, x);
    return DPZ_OK;
}

inline int id_bytes(int it) { return it == DPZ_I32 ? 4 : 8; }

// The bytes of one buffer of a call: `rows` rows of `width` bytes, `stride`
// bytes apart.
struct Block {
    const char* name;
    uintptr_t lo;
    int64_t rows, width, stride;
    bool written;
    uintptr_t hi() const { return lo + (rows - 1) * stride + width; }
};

inline Block mat_block(const char* name, const void* p, int64_t ld, int64_t rows, int64_t cols, int dt,
                bool written)
{
    const int es = elem_bytes(dt);
    return {name, reinterpret_cast<uintptr_t>(p), p ? rows : 0, cols * es, ld * es, written};
}

inline Block vec_block(const char* name, const void* p, int64_t bytes, bool written)
{
    return {name, reinterpret_cast<uintptr_t>(p), p && bytes > 0 ? 1 : 0, bytes, bytes, written};
}

// Whether two buffers share a byte.  Two matrices of one row stride may
// interleave, as column ranges of one larger matrix do.
inline bool overlap(const Block& a, const Block& b)
{
    if (a.rows < 1 || b.rows < 1 || a.lo >= b.hi() || b.lo >= a.hi()) return false;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
    const int64_t s = a.stride;
    const int64_t d = ((int64_t)(b.lo - a.lo) % s + s) % s;   // b's first column, from a's
    return !(a.width <= d && d + b.width <= s);
}

// No buffer that the call writes may share a byte with another one.
inline int check_blocks(std::initializer_list<Block> bs)
{
    for (const Block* a = bs.begin(); a != bs.end(); ++a)
        for (const Block* b = a + 1; b != bs.end(); ++b)
            if ((a->written || b->written) && overlap(*a, *b))
                return fail(DPZ_ERR_INVALID_ARG, "buffers %s and %s overlap", a->name, b->name);
    return DPZ_OK;
}

}  // namespace dpz
