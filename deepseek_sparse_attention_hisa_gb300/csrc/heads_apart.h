// Which strides of heads keep them apart. Plain C++, so that the host can check it.
#pragma once

#include <cstdint>

namespace hisa {

// Whether no two of an output's heads, of which `written` neighbouring elements are written, overlap: tokens lie
// `token` elements apart, a token's heads `head`. One layout nested in the other, as all but
// odd ones are, is seen at once.
inline bool heads_apart(int64_t tokens, int64_t heads, int64_t token, int64_t head, int64_t written) {
    if ((tokens > 1 && token < written) || (heads > 1 && head < written)) return false;
    if (tokens <= 1 || heads <= 1) return true;
    if (head / tokens >= token || token / heads >= head) return true;
    for (int64_t dh = 1; dh < heads; ++dh) {              // heads dh apart, of the tokens that come nearest
        const int64_t dt = dh * head / token;
        if (dt < tokens && dh * head - dt * token < written) return false;
        if (dt + 1 < tokens && (dt + 1) * token - dh * head < written) return false;
    }
    return true;
}

}  // namespace hisa
