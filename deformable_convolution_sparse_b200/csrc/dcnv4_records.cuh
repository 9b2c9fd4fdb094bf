// The record layout of the predictor's projection, as the operators around its
// weight read it.
#pragma once

namespace dcnv4 {

// Projection channel of slot s of a record of G groups of P points: a group's
// slots are its 2P offsets, then its P masks; the projection's channels are all
// groups' offsets, then all groups' masks.
__host__ __device__ __forceinline__ int slot_channel(int s, int G, int P) {
    const int g = s / (3 * P), r = s - g * 3 * P;
    return r < 2 * P ? g * 2 * P + r : 2 * G * P + g * P + (r - 2 * P);
}

}  // namespace dcnv4
